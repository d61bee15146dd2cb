// Norms of queries and keys for each head with the position rotation in the
// same pass, and their gradient, for sm_103a: the kernels (instantiated in
// rope_sm103.cu and rope_grad_sm103.cu).
//
// Both read and write every element once and are DRAM-bound.  A warp takes one
// token's heads of one block (of the queries or of the keys, UNROLL groups of
// heads at a time), a group of lanes a head; it keeps its frequencies and weights in registers
// and walks over tokens, and all loads of a token's block are in flight
// together.  A lane holds, of each vector pair it loads, both values of every
// rotated pair: vectors i and i + rot / 2 of the half layout, neighbouring
// vectors of the interleaved one, so that no value crosses lanes but the norm's sum.
//
// Angles: a frequency is kept as a 64-bit fixed-point number of turns, so that
// position * frequency, modulo 2^64, is the exact fraction of a turn at any
// position (in fp32 the product itself is off by 0.06 radians at position 10^6),
// in integer instructions rather than fp64 ones.
//
// Measured (GB300, 32768 tokens, 32 + 8 heads of 128, bf16, with norms): forward 107
// us, 6.3 TB/s; gradient 168 us, 6.0 TB/s, of which the weights' sums are 4 us.  Copy
// rate: 6.8 TB/s.
#pragma once

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "ptx.cuh"
#include "token_device.cuh"

namespace cdg {

struct RopeSide {           // queries or keys
    const void *x, *dy;     // dy: gradient only
    void *out;
    long long ld_x, ld_dy, ld_out;
    const float *w;         // NULL: ones
    float *dw;              // NULL: not wanted
    int heads, blocks, ctas;  // blocks of heads, CTAs a block
};

struct RopeArgs {
    RopeSide side[2];
    const void *positions;  // NULL: the token's number
    const float *inv_freq;
    float *partial;         // gradient: a row of dim sums for each CTA
    long long tokens;
    int index_bytes, dim, rot, interleaved, norm;
    int pairs;              // vector pairs of a head
    int lanes;              // a head's lanes: a power of two
    int block_heads;
    float factor, eps;
};

namespace {

constexpr int kMaxHead = 256, kMaxHeads = 65536;
constexpr int kRopeThreads = 256, kRopeWarps = kRopeThreads / 32;
// CTAs of a launch, at most: what 152 SMs hold at once (three an SM, two with the
// gradient's registers: 32768 x 40 heads of 128 took 107 and 168 us; with four and
// 64 registers 117, with three and 85 registers the gradient 176)
constexpr int kCtas = 456;
constexpr int kGradCtas = 304;

// Elements of a vector pair's two vectors: a and b the first of each, and
// whether the pair is rotated (half layout), or up to where (interleaved).
template <int V>
struct Pair {
    int a, b;
    bool turned;
    __device__ __forceinline__ Pair(const RopeArgs &p, int i)
    {
        const int n = p.interleaved ? 0 : p.rot / (2 * V);  // rotated vector pairs of the half layout
        turned = p.interleaved ? 2 * V * i < p.rot : i < n;
        a = i < n ? i * V : 2 * V * i;
        b = i < n ? p.rot / 2 + i * V : a + V;
    }
};

// V values as they lie in memory, and as fp32 pairs (one instruction for both;
// a single value is a pair with 0).
template <typename T, int V>
struct Raw {
    static constexpr int kBytes = V * static_cast<int>(sizeof(T)), kWords = kBytes < 4 ? 1 : kBytes / 4;
    static constexpr int kPacks = (V + 1) / 2;
    uint32_t w[kWords];
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0;
    }
    __device__ __forceinline__ void load(const T *src)
    {
        if constexpr (kBytes == 16) *reinterpret_cast<uint4 *>(w) = *reinterpret_cast<const uint4 *>(src);
        else if constexpr (kBytes == 8) *reinterpret_cast<uint2 *>(w) = *reinterpret_cast<const uint2 *>(src);
        else if constexpr (kBytes == 4) w[0] = *reinterpret_cast<const uint32_t *>(src);
        else w[0] = *reinterpret_cast<const uint16_t *>(src);
    }
    __device__ __forceinline__ void get(f32x2 (&f)[kPacks]) const
    {
        float g[2 * kPacks];
        g[2 * kPacks - 1] = 0.0f;
        if constexpr (kBytes >= 4) {
#pragma unroll
            for (int i = 0; i < kWords; ++i) widen<T>(w[i], g + i * kPerWord<T>);
        } else {
            widen<T>(w[0], g);
        }
#pragma unroll
        for (int i = 0; i < kPacks; ++i) f[i] = pack2(g[2 * i], g[2 * i + 1]);
    }
    __device__ __forceinline__ static void store(T *dst, const f32x2 (&f)[kPacks])
    {
        float g[2 * kPacks];
#pragma unroll
        for (int i = 0; i < kPacks; ++i) unpack2(f[i], g[2 * i], g[2 * i + 1]);
        if constexpr (kBytes < 4) {
            *dst = Elem<T>::put(g[0]);
        } else {
            uint32_t v[kWords];
#pragma unroll
            for (int i = 0; i < kWords; ++i) v[i] = narrow<T>(g + i * kPerWord<T>);
            if constexpr (kBytes == 16) *reinterpret_cast<uint4 *>(dst) = *reinterpret_cast<const uint4 *>(v);
            else if constexpr (kBytes == 8) *reinterpret_cast<uint2 *>(dst) = *reinterpret_cast<const uint2 *>(v);
            else *reinterpret_cast<uint32_t *>(dst) = v[0];
        }
    }
};

// f / (2 pi) turns, times 2^64, modulo 2^64: f's mantissa times 2^66 / (2 pi), shifted.
__device__ __forceinline__ uint64_t turns_of(float f)
{
    const uint64_t c = 0xA2F9836E4E441529ull;  // floor(2^66 / (2 pi)) = floor(2^65 / pi)
    const uint32_t bits = __float_as_uint(f);
    const int e = static_cast<int>((bits >> 23) & 255u);
    const uint64_t m = (bits & 0x7FFFFFu) | (e ? 0x800000u : 0u);
    const uint64_t lo = m * c, hi = __umul64hi(m, c);
    const int shift = (e ? e : 1) - 150 - 2;  // of the 128-bit product; below 0: to the right
    uint64_t t;
    if (shift <= -128) t = 0;
    else if (shift <= -64) t = hi >> (-shift - 64);
    else if (shift < 0) t = (lo >> -shift) | (hi << (64 + shift));
    else t = shift < 64 ? lo << shift : 0;
    return bits >> 31 ? 0ull - t : t;
}

// cos and sin of a fraction of a turn, times `factor`.  For 16-bit results the
// hardware's approximations (5e-7 off) do.
template <typename T>
__device__ __forceinline__ void cos_sin(uint64_t turn, float factor, float &c, float &s)
{
    if constexpr (sizeof(T) == 4) {
        const float x = static_cast<float>(static_cast<int64_t>(turn)) * 1.0842021724855044e-19f;  // 2^-63: half turns
        sincospif(x, &s, &c);
    } else {
        const float x = static_cast<float>(static_cast<int32_t>(turn >> 32)) * 1.4629180792671596e-9f;  // 2 pi / 2^32
        __sincosf(x, &s, &c);
    }
    c *= factor;
    s *= factor;
}

__device__ __forceinline__ int64_t position_of(const RopeArgs &p, long long token)
{
    if (!p.positions) return token;
    return p.index_bytes == 8 ? __ldg(static_cast<const long long *>(p.positions) + token)
                              : __ldg(static_cast<const int *>(p.positions) + token);
}

// (a, b) turned by the angles of (c, s).  In the interleaved layout the pairs
// lie within a, then within b.
template <int V>
__device__ __forceinline__ void turn(bool interleaved, const float (&c)[V], const float (&s)[V], f32x2 (&a)[(V + 1) / 2], f32x2 (&b)[(V + 1) / 2])
{
    if (V > 1 && interleaved) {
#pragma unroll
        for (int i = 0; i < (V + 1) / 2; ++i) {
            const int j = (V / 2 + i) % V;  // b's angles follow a's
            float x, y;
            unpack2(a[i], x, y);
            a[i] = fma2(pack2(y, x), pack2(-s[i], s[i]), mul2(a[i], pack2(c[i], c[i])));
            unpack2(b[i], x, y);
            b[i] = fma2(pack2(y, x), pack2(-s[j], s[j]), mul2(b[i], pack2(c[j], c[j])));
        }
    } else {
#pragma unroll
        for (int i = 0; i < (V + 1) / 2; ++i) {
            const int j = V > 1 ? 2 * i + 1 : 0;
            const f32x2 cc = pack2(c[(2 * i) % V], c[j]), u = a[i];
            a[i] = fma2(b[i], pack2(-s[(2 * i) % V], -s[j]), mul2(u, cc));
            b[i] = fma2(u, pack2(s[(2 * i) % V], s[j]), mul2(b[i], cc));
        }
    }
}

// GRAD: dx from dy and (with the norm) x, and the sums for dw.  A lane has R
// vector pairs.  LANES > 0: the head is 2 V LANES values, a lane has one whole
// pair, and the layout is INTERLEAVED or not; 0: whatever the call says.
//
// Issue-bound before that (177 instructions for two heads of 128: bounds of every
// lane and head, addresses, a loop of shuffles): what a size fixes is fixed when
// the kernel is compiled, and a block's last heads alone are checked.
template <typename T, int V, int UNROLL, bool GRAD, bool NORM, bool INTERLEAVED, int LANES>
__global__ void __launch_bounds__(kRopeThreads, !GRAD || !NORM ? 3 : 2) rope_kernel(const __grid_constant__ RopeArgs p)
{
    constexpr int R = V >= 4 ? 1 : 4 / V, N = (V + 1) / 2;
    constexpr bool X = !GRAD || NORM;  // whether x is read
    __shared__ float red[GRAD && NORM ? kRopeWarps : 1][GRAD && NORM ? kMaxHead : 1];
    grid_dep_launch_dependents();
    grid_dep_wait();
    const int lanes = LANES ? LANES : p.lanes, dim = LANES ? 2 * V * LANES : p.dim;
    const bool interleaved = LANES ? INTERLEAVED : p.interleaved != 0;
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    // this CTA's side, block of heads, and place among the block's CTAs
    int cta = blockIdx.x;
    const bool keys = cta >= p.side[0].blocks * p.side[0].ctas;
    const RopeSide &sd = p.side[keys];
    if (keys) cta -= p.side[0].blocks * p.side[0].ctas;
    const int block = cta / sd.ctas, part = cta - block * sd.ctas;
    const int groups = 32 / lanes, group = lane / lanes, l = lane - group * lanes;
    const int h_first = block * p.block_heads, h_end = min(sd.heads, h_first + p.block_heads);

    int at_a[R], at_b[R];
    bool has_a[R], has_b[R], turned[R];
    uint64_t freq[R][V];
    // An infinite or NaN frequency is no number of turns, and its angles are NaN: carried by the
    // factor, that reaches all of this lane's pairs (a check of every pair of every token cost 3 %).
    float factor = p.factor;
    f32x2 wa[R][N], wb[R][N], dwa[R][N], dwb[R][N];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const Pair<V> v(p, l + i * 32);
        at_a[i] = v.a;
        at_b[i] = v.b;
        turned[i] = v.turned;
        has_a[i] = LANES || (l + i * 32 < p.pairs && v.a < dim);
        has_b[i] = LANES || (has_a[i] && v.b < dim);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            // rotated pairs' numbers: those of the vector pair; past the rotated part the angle is 0
            const int k = interleaved ? v.a / 2 + e : v.a + e;
            const float f = turned[i] && 2 * k < p.rot ? __ldg(p.inv_freq + k) : 0.0f;
            freq[i][e] = turns_of(f);
            if (!isfinite(f)) factor = __int_as_float(0x7FC00000);
        }
#pragma unroll
        for (int e = 0; e < N; ++e) {
            auto weight = [&](bool has, int at, bool second) {
                return second && V == 1 ? 0.0f : sd.w && has ? __ldg(sd.w + at + 2 * e + second) : 1.0f;
            };
            wa[i][e] = pack2(weight(has_a[i], v.a, false), weight(has_a[i], v.a, true));
            wb[i][e] = pack2(weight(has_b[i], v.b, false), weight(has_b[i], v.b, true));
            dwa[i][e] = dwb[i][e] = pack2(0.0f, 0.0f);
        }
    }
    const bool all_turned = p.rot == dim;
    const float inv_dim = 1.0f / static_cast<float>(dim);
    float c[R][V], s[R][V];

    // UNROLL groups' heads from hb of one token; WHOLE: all of them are the block's.
    // The rows' pointers are those of this lane in the batch's first group.
    auto batch = [&](auto whole, const T *x, const T *dy, T *out, int left, long long token, bool first) {
        constexpr bool WHOLE = decltype(whole)::value;
        Raw<T, V> xa[X ? UNROLL : 1][R], xb[X ? UNROLL : 1][R], ya[GRAD ? UNROLL : 1][R], yb[GRAD ? UNROLL : 1][R];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const int row = u * groups * dim;
            const bool in = WHOLE || u * groups + group < left;
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const bool in_a = in && has_a[i], in_b = in && has_b[i];
                if (X) {
                    if (!WHOLE || !LANES) xa[u][i].clear(), xb[u][i].clear();
                    if (in_a) xa[u][i].load(x + row + at_a[i]);
                    if (in_b) xb[u][i].load(x + row + at_b[i]);
                }
                if (GRAD) {
                    if (!WHOLE || !LANES) ya[u][i].clear(), yb[u][i].clear();
                    if (in_a) ya[u][i].load(dy + row + at_a[i]);
                    if (in_b) yb[u][i].load(dy + row + at_b[i]);
                }
            }
        }
        if (first) {  // (beneath the first loads)
            const uint64_t pos = static_cast<uint64_t>(position_of(p, token));
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const int k = interleaved ? at_a[i] / 2 + e : at_a[i] + e;
                    if (all_turned || (turned[i] && 2 * k < p.rot)) cos_sin<T>(pos * freq[i][e], factor, c[i][e], s[i][e]);
                    else c[i][e] = 1.0f, s[i][e] = 0.0f;
                    if (GRAD) s[i][e] = -s[i][e];  // back
                }
        }
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            if (!WHOLE && u * groups >= left) break;  // (the same for the whole warp)
            f32x2 fa[R][N], fb[R][N], ga[R][N], gb[R][N];  // x, and the gradient dz
            f32x2 sum = pack2(0.0f, 0.0f), dot = sum;
#pragma unroll
            for (int i = 0; i < R; ++i) {
                if (X) {
                    xa[u][i].get(fa[i]);
                    xb[u][i].get(fb[i]);
                }
                if (GRAD) {
                    ya[u][i].get(ga[i]);
                    yb[u][i].get(gb[i]);
                    if (all_turned || turned[i]) turn<V>(interleaved, c[i], s[i], ga[i], gb[i]);
                }
                if (NORM) {
#pragma unroll
                    for (int e = 0; e < N; ++e) {
                        sum = fma2(fa[i][e], fa[i][e], sum);
                        sum = fma2(fb[i][e], fb[i][e], sum);
                        if (GRAD) {
                            dot = fma2(mul2(ga[i][e], wa[i][e]), fa[i][e], dot);
                            dot = fma2(mul2(gb[i][e], wb[i][e]), fb[i][e], dot);
                        }
                    }
                }
            }
            f32x2 scale, back;  // 1 / sqrt(mean(x^2) + eps), and - mean(dn n) times it
            if (NORM) {
                float q, q1, g, g1;
                unpack2(sum, q, q1);
                unpack2(dot, g, g1);
                q += q1;
                g += g1;
#pragma unroll
                for (int d = 16; d; d /= 2)
                    if (d < lanes) {
                        q += __shfl_xor_sync(0xFFFFFFFFu, q, d);
                        if (GRAD) g += __shfl_xor_sync(0xFFFFFFFFu, g, d);
                    }
                q = rsqrtf(fmaf(q, inv_dim, p.eps));
                // (a head past the last has x = dz = 0 and, with eps = 0, no finite scale of its own)
                if (GRAD && !WHOLE && u * groups + group >= left) q = 0.0f;
                scale = pack2(q, q);
                if (GRAD) {
                    g = -(q * q * (g * inv_dim));
                    back = pack2(g, g);
                }
            }
            const bool in = WHOLE || u * groups + group < left;
#pragma unroll
            for (int i = 0; i < R; ++i) {
                if (NORM) {
#pragma unroll
                    for (int e = 0; e < N; ++e) {
                        if (!GRAD) {
                            fa[i][e] = mul2(fa[i][e], mul2(scale, wa[i][e]));
                            fb[i][e] = mul2(fb[i][e], mul2(scale, wb[i][e]));
                        } else {
                            // (a head past the last has dz = x = scale = 0)
                            dwa[i][e] = fma2(ga[i][e], mul2(fa[i][e], scale), dwa[i][e]);
                            dwb[i][e] = fma2(gb[i][e], mul2(fb[i][e], scale), dwb[i][e]);
                            ga[i][e] = mul2(scale, fma2(fa[i][e], back, mul2(ga[i][e], wa[i][e])));
                            gb[i][e] = mul2(scale, fma2(fb[i][e], back, mul2(gb[i][e], wb[i][e])));
                        }
                    }
                }
                if (!GRAD && (all_turned || turned[i])) turn<V>(interleaved, c[i], s[i], fa[i], fb[i]);
                const int row = u * groups * dim;
                if (in && has_a[i]) Raw<T, V>::store(out + row + at_a[i], GRAD ? ga[i] : fa[i]);
                if (in && has_b[i]) Raw<T, V>::store(out + row + at_b[i], GRAD ? gb[i] : fb[i]);
            }
        }
    };
    const long long stride = static_cast<long long>(sd.ctas) * kRopeWarps;
    const int head0 = (h_first + group) * dim, step = UNROLL * groups * dim;  // (heads * dim is below 2^24)
    for (long long token = static_cast<long long>(part) * kRopeWarps + warp; token < p.tokens; token += stride) {
        const T *x = X ? static_cast<const T *>(sd.x) + token * sd.ld_x + head0 : nullptr;
        const T *dy = GRAD ? static_cast<const T *>(sd.dy) + token * sd.ld_dy + head0 : nullptr;
        T *out = static_cast<T *>(sd.out) + token * sd.ld_out + head0;
        for (int left = h_end - h_first; left > 0; left -= UNROLL * groups) {
            const bool first = left == h_end - h_first;
            if (left >= UNROLL * groups) batch(std::true_type{}, x, dy, out, left, token, first);
            else batch(std::false_type{}, x, dy, out, left, token, first);
            if (X) x += step;
            if (GRAD) dy += step;
            out += step;
        }
    }
    if (GRAD && NORM && sd.dw) {
        // a warp's groups of lanes, then the CTA's warps, in order
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                float a[2], b[2];
                unpack2(dwa[i][e / 2], a[0], a[1]);
                unpack2(dwb[i][e / 2], b[0], b[1]);
                float va = a[e & 1], vb = b[e & 1];
                for (int d = lanes; d < 32; d *= 2) {
                    va += __shfl_xor_sync(0xFFFFFFFFu, va, d);
                    vb += __shfl_xor_sync(0xFFFFFFFFu, vb, d);
                }
                if (group == 0 && has_a[i]) red[warp][at_a[i] + e] = va;
                if (group == 0 && has_b[i]) red[warp][at_b[i] + e] = vb;
            }
        __syncthreads();
        for (int d = threadIdx.x; d < dim; d += kRopeThreads) {
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < kRopeWarps; ++w) v += red[w][d];
            p.partial[static_cast<long long>(blockIdx.x) * dim + d] = v;
        }
    }
}

// Vector width: the widest at which every vector of every row starts on its own
// size and no rotated half, nor the head, ends inside one.
template <typename T>
int vector_width(const RopeArgs &a, bool grad)
{
    for (int v = 4; v > 1; v /= 2) {
        bool fits = a.dim % v == 0 && a.rot % (a.interleaved ? 2 : 2 * v) == 0;
        for (const RopeSide &s : a.side) {
            if (s.heads == 0) continue;
            const size_t bytes = v * sizeof(T);
            if (!grad || a.norm) fits = fits && aligned_to(s.x, bytes) && s.ld_x % v == 0;
            if (grad) fits = fits && aligned_to(s.dy, bytes) && s.ld_dy % v == 0;
            fits = fits && aligned_to(s.out, bytes) && s.ld_out % v == 0;
        }
        if (fits) return v;
    }
    return 1;
}

template <typename T, int V, bool GRAD, bool NORM>
cudaError_t launch_width(RopeArgs &a, cudaStream_t s)
{
    constexpr int UNROLL = V == 4 ? 4 : 2;
    const int n = a.interleaved ? (a.dim + 2 * V - 1) / (2 * V) : a.rot / (2 * V) + (a.dim - a.rot + 2 * V - 1) / (2 * V);
    a.pairs = n;
    a.lanes = 1;
    while (a.lanes < 32 && a.lanes < n) a.lanes *= 2;
    const int heads = a.side[0].heads + a.side[1].heads;
    // two batches a block where the tokens alone give every warp work: the angles are computed once a block
    a.block_heads = 32 / a.lanes * UNROLL;
    if (a.tokens >= kCtas * kRopeWarps) a.block_heads *= 2;
    // a block's CTAs in proportion to its side's heads
    const long long most = (a.tokens + kRopeWarps - 1) / kRopeWarps;
    long long ctas = 0;
    for (RopeSide &sd : a.side) {
        sd.blocks = (sd.heads + a.block_heads - 1) / a.block_heads;
        if (sd.blocks == 0) continue;
        const long long share = static_cast<long long>(GRAD ? kGradCtas : kCtas) * sd.heads / heads / sd.blocks;
        sd.ctas = static_cast<int>(std::max(1ll, std::min(most, share)));
        ctas += static_cast<long long>(sd.blocks) * sd.ctas;
    }
    const dim3 grid(static_cast<unsigned>(ctas)), block(kRopeThreads);
    if constexpr (V == 4) {
        if (a.dim == 2 * V * a.pairs && (a.pairs == 16 || a.pairs == 8)) {
            void (*k)(RopeArgs) = a.interleaved ? (a.pairs == 16 ? rope_kernel<T, V, UNROLL, GRAD, NORM, true, 16> : rope_kernel<T, V, UNROLL, GRAD, NORM, true, 8>)
                                                : (a.pairs == 16 ? rope_kernel<T, V, UNROLL, GRAD, NORM, false, 16> : rope_kernel<T, V, UNROLL, GRAD, NORM, false, 8>);
            return launch_early(k, grid, block, 0, s, a);
        }
    }
    return launch_early(rope_kernel<T, V, UNROLL, GRAD, NORM, false, 0>, grid, block, 0, s, a);
}

template <typename T, bool GRAD>
cudaError_t launch_rope(RopeArgs &a, cudaStream_t s)
{
    switch (vector_width<T>(a, GRAD)) {
    case 4: return a.norm ? launch_width<T, 4, GRAD, true>(a, s) : launch_width<T, 4, GRAD, false>(a, s);
    case 2: return a.norm ? launch_width<T, 2, GRAD, true>(a, s) : launch_width<T, 2, GRAD, false>(a, s);
    default: return a.norm ? launch_width<T, 1, GRAD, true>(a, s) : launch_width<T, 1, GRAD, false>(a, s);
    }
}

}  // namespace
}  // namespace cdg

// the gradient's kernels and the sum of their partial rows, in rope_grad_sm103.cu
cudaError_t crp_launch_grad(cdg::RopeArgs &a, int dtype, cudaStream_t s);
