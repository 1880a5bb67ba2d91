// Attention of prompts over keys and values expanded from latents
// (hr_latent_prompt_attention).
//
// Mathematics.  Softmax attention in one pass: a running reference m, the sum of
// exp(w - m), and the sums of exp(w - m) v.  The reference only has to keep the
// exponentials in range, so it moves when one passes 2^kFar, and everything is
// rescaled then.  A key is a part of its head's own and the rotary key that all
// heads share, which meets the other in LDS.
//
// Layout.  A workgroup takes kRows query rows of one head of a sequence, 16 RT to a
// wave, and passes over the keys 64 at a time, which all waves share in LDS; the
// next 64 are on their way in registers meanwhile.  Scores are formed transposed,
// S^T = K Q^T (A operand: keys, B operand: queries, in registers throughout), so that
// a lane holds four keys of one row, and two tiles of 16 keys are as they stand the B
// operand of O^T = V^T P^T, with V^T out of LDS by transposing reads: probabilities
// never leave the registers.  Operands are bfloat16 and sums float32: a probability is
// rounded to 8 bits, since the values may lie anywhere in bfloat16's range, which float16
// has not, and both operands of a product are of one type; the sum that divides them is
// of the unrounded ones.  A chunk errs by 2.3e-3 of its norm, where the result's own
// rounding makes 1.7e-3.
//
// Measured: a chunk of 2048 tokens behind 6144 positions, 32 heads of 128 + 64 (301
// GFLOP), in 329 us, 915 TFLOP/s, three quarters of what a large bfloat16 product
// reaches here; three ragged prompts of up to 777, 16 heads, in 34 us: 160 workgroups, one
// wave a SIMD, and the longest prompt's last rows with 13 steps of 2.6 us in a row.
// Exponentials and the reads of keys and values from LDS stand beside the matrix steps of
// two waves a SIMD (of the chunk's cycles 38% are matrix instructions, 42% vector ones, and
// LDS is active for 40%, 11% of them conflicts); registers leave no room for a third with
// 32 rows a wave, and with 16 each the reads are twice as many.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "latent.h"

namespace hr {
namespace {

typedef uint32_t uint4v __attribute__((ext_vector_type(4)));
typedef uint32_t uint2v __attribute__((ext_vector_type(2)));
typedef __bf16 bfloat8 __attribute__((ext_vector_type(8)));
typedef __bf16 bfloat2 __attribute__((ext_vector_type(2)));
typedef float float4v __attribute__((ext_vector_type(4)));
typedef short short4v __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLow = -3.0e38f;      // reference of a row that has seen nothing
constexpr float kFar = 0x1p8f;        // largest exponential before the reference moves
constexpr int kKeys = 64;             // of a step
constexpr int kWaves = 4;

__device__ __forceinline__ float4v mfma(uint4v a, uint4v b, float4v c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bfloat8, a), __builtin_bit_cast(bfloat8, b), c, 0, 0, 0);
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    bfloat2 h;
    h.x = static_cast<__bf16>(a);
    h.y = static_cast<__bf16>(b);
    return __builtin_bit_cast(uint32_t, h);
}
__device__ __forceinline__ float max_groups(float v) {
    v = fmaxf(v, __shfl_xor(v, 16));
    return fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float sum_groups(float v) {
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}
// 16 dimensions of four keys out of LDS: lane m of 16 gives the address of its four
// dimensions 4 (m % 4) of key m / 4, and gets dimension m of the four keys
__device__ __forceinline__ uint2v transposed(const uint8_t* p) {
    typedef short4v __attribute__((address_space(3)))* Lds;
    return __builtin_bit_cast(uint2v, __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)(p)));
}
// whether a bfloat16 of two is infinite or NaN
__device__ __forceinline__ bool odd_pair(uint32_t x) {
    return (x & 0x7F800000u) == 0x7F800000u || (x & 0x7F80u) == 0x7F80u;
}
__device__ __forceinline__ uint32_t finite_pair(uint32_t x) {
    if ((x & 0x7F800000u) == 0x7F800000u) x &= 0xFFFFu;
    if ((x & 0x7F80u) == 0x7F80u) x &= 0xFFFF0000u;
    return x;
}

__device__ __forceinline__ int clamped(const int32_t* cu, int b, int most) { return min(max(cu[b], 0), most); }

template <int N, int RT>
__global__ void __launch_bounds__(64 * kWaves, 2) latent_prompt(const LatentPromptArgs a) {
    constexpr int M = 16 * RT * kWaves;
    constexpr int KS = (N + kRope) / 32, DT = N / 16, KT = kKeys / 16;
    constexpr int KB = 2 * (N + kRope) + 16, VB = 2 * N + 32;   // bytes of a key and a value in LDS
    constexpr int KL = kKeys * N / 8 / (64 * kWaves), RL = kKeys * kRope / 8 / (64 * kWaves);   // 16-byte loads of a thread
    __shared__ __attribute__((aligned(16))) uint8_t keys[kKeys * KB];
    __shared__ __attribute__((aligned(16))) uint8_t values[kKeys * VB];
    __shared__ uint32_t odd[kKeys / 32];       // values that are not finite, by key
    const int tid = threadIdx.x, lane = tid & 63, m = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int h = blockIdx.x % a.heads, u = blockIdx.x / a.heads;
    // the last sequence b with floor(cu(b) / M) + b <= u, a bound that leaves every
    // sequence at least the blocks it needs
    int lo = 0, hi = a.rows - 1;
    while (lo < hi) {
        const int mid = lo + (hi - lo + 1) / 2;
        if (clamped(a.cu_q, mid, a.tokens) / M + mid <= u) lo = mid;
        else hi = mid - 1;
    }
    const int start = clamped(a.cu_q, lo, a.tokens), n = max(clamped(a.cu_q, lo + 1, a.tokens) - start, 0);
    const int k_start = clamped(a.cu_k, lo, a.positions), len = max(clamped(a.cu_k, lo + 1, a.positions) - k_start, 0);
    const int blocks = (n + M - 1) / M, nth = u - (start / M + lo);
    if (nth >= blocks) return;
    const int r0 = (blocks - 1 - nth) * M;     // (rows that see most come first)
    const int first = len - n;                 // position of the first token (may lie before 0)

    uint4v query[RT][KS];
    int pos[RT];                               // the last key that the lane's row sees
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        const int r = min(r0 + (wave * RT + rt) * 16 + m, n - 1);
        const uint16_t* q = a.q + (static_cast<int64_t>(start) + r) * a.q_st + h * a.q_sh;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) query[rt][ks] = *reinterpret_cast<const uint4v*>(q + 32 * ks + 8 * g);
        pos[rt] = a.causal ? min(first + r, len - 1) : len - 1;
    }
    const int limit = a.causal ? min(max(first + min(r0 + M, n), 0), len) : len;
    const int all = a.causal ? min(first + min(r0 + wave * 16 * RT, n - 1) + 1, len) : len;   // all of the wave's rows see keys below
    const int every = a.causal ? min(first + r0 + 1, len) : len;                              // all of the workgroup's rows

    float4v acc[RT][DT];
    float ref[RT], sum[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        ref[rt] = kLow;
        sum[rt] = 0.0f;
#pragma unroll
        for (int d = 0; d < DT; ++d) acc[rt][d] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
    }
    const float factor = a.scale * kLog2e;

    uint4v kn[KL], vn[KL], rn[RL];             // the next keys
    const auto load = [&](int t0) {
#pragma unroll
        for (int i = 0; i < KL; ++i) {
            const int x = i * 64 * kWaves + tid, j = x / (N / 8), c = x % (N / 8) * 8;
            const int64_t at = k_start + static_cast<int64_t>(min(t0 + j, len - 1));
            kn[i] = *reinterpret_cast<const uint4v*>(a.k + at * a.k_st + h * a.k_sh + c);
            vn[i] = *reinterpret_cast<const uint4v*>(a.v + at * a.v_st + h * a.v_sh + c);
        }
#pragma unroll
        for (int i = 0; i < RL; ++i) {
            const int x = i * 64 * kWaves + tid, j = x / (kRope / 8), c = x % (kRope / 8) * 8;
            rn[i] = *reinterpret_cast<const uint4v*>(a.rope + (k_start + static_cast<int64_t>(min(t0 + j, len - 1))) * a.r_st + c);
        }
    };
    if (limit > 0) load(0);
    for (int t0 = 0; t0 < limit; t0 += kKeys) {
        // What a row does not see must not reach it, and 0 times an infinite or NaN
        // value would: where not every row sees every key such values are taken out,
        // and added apart for the rows that see them.
        const bool masked = t0 + kKeys > every;
        __syncthreads();                       // (the last step's readers are done)
        if (tid < kKeys / 32) odd[tid] = 0;
        if (masked) __syncthreads();
#pragma unroll
        for (int i = 0; i < KL; ++i) {
            const int x = i * 64 * kWaves + tid, j = x / (N / 8), c = x % (N / 8) * 16;
            *reinterpret_cast<uint4v*>(keys + j * KB + c) = kn[i];
            uint4v v = vn[i];
            if (masked) {
                if (t0 + j >= len) v = uint4v{0, 0, 0, 0};
                if (odd_pair(v.x) || odd_pair(v.y) || odd_pair(v.z) || odd_pair(v.w)) {
                    atomicOr(&odd[j / 32], 1u << (j % 32));
#pragma unroll
                    for (int y = 0; y < 4; ++y) v[y] = finite_pair(v[y]);
                }
            }
            *reinterpret_cast<uint4v*>(values + j * VB + c) = v;
        }
#pragma unroll
        for (int i = 0; i < RL; ++i) {
            const int x = i * 64 * kWaves + tid, j = x / (kRope / 8), c = x % (kRope / 8) * 16;
            *reinterpret_cast<uint4v*>(keys + j * KB + 2 * N + c) = rn[i];
        }
        __syncthreads();
        if (t0 + kKeys < limit) load(t0 + kKeys);

        // scores
        float4v w[RT][KT];
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) w[rt][kt] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                const uint4v k = *reinterpret_cast<const uint4v*>(keys + (16 * kt + m) * KB + 64 * ks + 16 * g);
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) w[rt][kt] = mfma(k, query[rt][ks], w[rt][kt]);
            }
        }
        if (t0 + kKeys > all) {
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (t0 + 16 * kt + 4 * g + i > pos[rt]) w[rt][kt][i] = -__builtin_inff();
        }
        // exponentials; the reference moves where one is too large
        uint4v p[RT][KT / 2];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            float e[KT][4], l = 0.0f;
            const auto exps = [&]() {
                bool far = false;
                l = 0.0f;
#pragma unroll
                for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        e[kt][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(w[rt][kt][i], factor, -ref[rt]));
                        far = far || !(e[kt][i] <= kFar);
                        l += e[kt][i];
                    }
                return far;
            };
            if (__any(exps())) {
                float x = w[rt][0][0];
#pragma unroll
                for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) x = fmaxf(x, w[rt][kt][i]);
                x = max_groups(x) * factor;
                const float was = ref[rt];
                if (x < __builtin_inff()) ref[rt] = fmaxf(was, x);
                const float f = __builtin_amdgcn_exp2f(was - ref[rt]);
                sum[rt] *= f;
#pragma unroll
                for (int d = 0; d < DT; ++d)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[rt][d][i] *= f;
                exps();
            }
            sum[rt] += l;
#pragma unroll
            for (int k = 0; k < KT / 2; ++k)
                p[rt][k] = uint4v{pack_bf16(e[2 * k][0], e[2 * k][1]), pack_bf16(e[2 * k][2], e[2 * k][3]),
                                  pack_bf16(e[2 * k + 1][0], e[2 * k + 1][1]), pack_bf16(e[2 * k + 1][2], e[2 * k + 1][3])};
        }
        // sums
        const uint8_t* va = values + (4 * g + m / 4) * VB + 8 * (m % 4);
#pragma unroll
        for (int k = 0; k < KT / 2; ++k)
#pragma unroll
            for (int d = 0; d < DT; ++d) {
                const uint2v v0 = transposed(va + (32 * k) * VB + 32 * d), v1 = transposed(va + (32 * k + 16) * VB + 32 * d);
                const uint4v v = {v0.x, v0.y, v1.x, v1.y};
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) acc[rt][d] = mfma(v, p[rt][k], acc[rt][d]);
            }
        if (masked && (odd[0] | odd[1])) {
            // rare: the values that were taken out, for the rows that see them
            for (int j = 0; j < kKeys; ++j) {
                if (!((odd[j / 32] >> (j % 32)) & 1)) continue;
                const uint16_t* v = a.v + (k_start + static_cast<int64_t>(t0 + j)) * a.v_st + h * a.v_sh;
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    // the row's probability of key j, from the lane that has it
                    const int word = (j & 16) / 8 + (j & 2) / 2;
                    uint32_t x = 0;
#pragma unroll
                    for (int k = 0; k < KT / 2; ++k)
#pragma unroll
                        for (int y = 0; y < 4; ++y) x = k == j / 32 && y == word ? p[rt][k][y] : x;
                    x = __shfl(x, m + 16 * ((j & 15) / 4));
                    const float e = __uint_as_float((j & 1) ? x & 0xFFFF0000u : x << 16);
                    if (t0 + j <= pos[rt]) {
#pragma unroll
                        for (int d = 0; d < DT; ++d)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const uint32_t b = v[16 * d + 4 * g + i];
                                if ((b & 0x7F80u) == 0x7F80u) acc[rt][d][i] += e * __uint_as_float(b << 16);
                            }
                    }
                }
            }
        }
    }
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        const int r = r0 + (wave * RT + rt) * 16 + m;
        const float l = sum_groups(sum[rt]), inverse = 1.0f / l;
        if (r >= n) continue;
        uint16_t* out = a.out + (static_cast<int64_t>(start) + r) * a.o_st + h * a.o_sh;
#pragma unroll
        for (int d = 0; d < DT; ++d) {
            float4v v = acc[rt][d];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = l == 0.0f ? 0.0f : v[i] * inverse;
            *reinterpret_cast<uint2v*>(out + 16 * d + 4 * g) = uint2v{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
        }
        if (a.lse && g == 0)
            a.lse[(static_cast<int64_t>(start) + r) * a.heads + h] =
                l == 0.0f ? -__builtin_inff() : (ref[rt] + __builtin_amdgcn_logf(l)) * 0.6931471805599453f;
    }
}

template <int N, int RT>
void prompt_launch(const LatentPromptArgs& a, hipStream_t s) {
    const int64_t blocks = int64_t{a.tokens} / (16 * RT * kWaves) + a.rows;
    hipLaunchKernelGGL((latent_prompt<N, RT>), dim3(static_cast<uint32_t>(blocks * a.heads)), dim3(64 * kWaves), 0, s, a);
}

}  // namespace

int launch_latent_prompt(const LatentPromptArgs& a, void* stream) {
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (a.nope == 128) prompt_launch<128, 2>(a, s);
    else prompt_launch<64, 2>(a, s);
    return static_cast<int>(hipGetLastError());
}

}  // namespace hr
