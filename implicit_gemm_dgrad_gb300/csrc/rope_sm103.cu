// Norms of queries and keys for each head with the position rotation in the
// same pass, and their gradient, for sm_103a: kernels and C entry points.
//
// Both read and write every element once and are DRAM-bound.  A warp takes one
// token's heads of one block (queries or keys, up to kUnroll groups of heads),
// a group of lanes a head; it keeps its frequencies and weights in registers
// and walks over tokens, and all loads of a token's block are in flight
// together.  A lane holds, of each vector pair it loads, both values of every
// rotated pair: vectors i and i + rot / 2 of the half layout, neighbouring
// vectors of the interleaved one, so that no value crosses lanes but the norm's sum.
//
// Angles: a frequency is kept as a 64-bit fixed-point number of turns, so that
// position * frequency, modulo 2^64, is the exact fraction of a turn at any
// position (in fp32 the product itself is off by 0.06 radians at position 10^6),
// in integer instructions rather than fp64 ones.
#include <algorithm>
#include <cmath>

#include "ptx.cuh"
#include "token_device.cuh"

namespace cdg {
namespace {

constexpr int kMaxHead = 256, kMaxHeads = 65536;
constexpr int kRopeThreads = 256, kRopeWarps = kRopeThreads / 32;
constexpr int kCtas = 1216;    // of a launch, at most: 8 an SM
constexpr int kGradCtas = 608;

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
template <int V, bool INTERLEAVED>
__device__ __forceinline__ void turn(const float (&c)[V], const float (&s)[V], f32x2 (&a)[(V + 1) / 2], f32x2 (&b)[(V + 1) / 2])
{
#pragma unroll
    for (int i = 0; i < (V + 1) / 2; ++i) {
        if constexpr (V > 1 && INTERLEAVED) {
            const int j = V / 2 + i;  // b's angles follow a's
            float x, y;
            unpack2(a[i], x, y);
            a[i] = fma2(pack2(y, x), pack2(-s[i], s[i]), mul2(a[i], pack2(c[i], c[i])));
            unpack2(b[i], x, y);
            b[i] = fma2(pack2(y, x), pack2(-s[j], s[j]), mul2(b[i], pack2(c[j], c[j])));
        } else {
            const int j = V > 1 ? 2 * i + 1 : 0;
            const f32x2 cc = pack2(c[2 * i], c[j]), u = a[i];
            a[i] = fma2(b[i], pack2(-s[2 * i], -s[j]), mul2(u, cc));
            b[i] = fma2(u, pack2(s[2 * i], s[j]), mul2(b[i], cc));
        }
    }
}

// GRAD: dx from dy and (with the norm) x, and the sums for dw.  A lane has R
// vector pairs; FULL: every lane has its one, whole.
template <typename T, int V, int UNROLL, bool GRAD, bool NORM, bool INTERLEAVED, bool FULL>
__global__ void __launch_bounds__(kRopeThreads, !GRAD ? 4 : NORM ? 2 : 3) rope_kernel(const __grid_constant__ RopeArgs p)
{
    constexpr int R = V >= 4 ? 1 : 4 / V, N = (V + 1) / 2;
    constexpr bool X = !GRAD || NORM;  // whether x is read
    __shared__ float red[GRAD && NORM ? kRopeWarps : 1][GRAD && NORM ? kMaxHead : 1];
    grid_dep_launch_dependents();
    grid_dep_wait();
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    // this CTA's side, block of heads, and place among the block's CTAs
    int cta = blockIdx.x;
    const bool keys = cta >= p.side[0].blocks * p.side[0].ctas;
    const RopeSide &sd = p.side[keys];
    if (keys) cta -= p.side[0].blocks * p.side[0].ctas;
    const int block = cta / sd.ctas, part = cta - block * sd.ctas;
    const int groups = 32 / p.lanes, group = lane / p.lanes, l = lane - group * p.lanes;
    const int h0 = block * p.block_heads + group, h_end = min(sd.heads, (block + 1) * p.block_heads);

    int at_a[R], at_b[R];
    bool has_a[R], has_b[R], turned[R];
    uint64_t freq[R][V];
    f32x2 wa[R][N], wb[R][N], dwa[R][N], dwb[R][N];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const Pair<V> v(p, l + i * 32);
        at_a[i] = v.a;
        at_b[i] = v.b;
        turned[i] = v.turned;
        has_a[i] = FULL || (l + i * 32 < p.pairs && v.a < p.dim);
        has_b[i] = FULL || (has_a[i] && v.b < p.dim);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            // rotated pairs' numbers: those of the vector pair; past the rotated part the angle is 0
            const int k = INTERLEAVED ? v.a / 2 + e : v.a + e;
            freq[i][e] = turned[i] && 2 * k < p.rot ? turns_of(__ldg(p.inv_freq + k)) : 0;
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
    const bool all_turned = p.rot == p.dim;
    const float inv_dim = 1.0f / static_cast<float>(p.dim);
    for (long long token = static_cast<long long>(part) * kRopeWarps + warp; token < p.tokens;
         token += static_cast<long long>(sd.ctas) * kRopeWarps) {
        const T *x = static_cast<const T *>(sd.x) + token * sd.ld_x, *dy = static_cast<const T *>(sd.dy) + token * sd.ld_dy;
        T *out = static_cast<T *>(sd.out) + token * sd.ld_out;
        float c[R][V], s[R][V];
        bool first = true;
        for (int hb = h0; hb - group < h_end; hb += UNROLL * groups) {
            Raw<T, V> xa[X ? UNROLL : 1][R], xb[X ? UNROLL : 1][R], ya[GRAD ? UNROLL : 1][R], yb[GRAD ? UNROLL : 1][R];
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) {
                const int h = hb + u * groups, row = h * p.dim;  // (heads * dim is below 2^24)
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    if (X) {
                        xa[u][i].clear();
                        xb[u][i].clear();
                        if (h < h_end && has_a[i]) xa[u][i].load(x + row + at_a[i]);
                        if (h < h_end && has_b[i]) xb[u][i].load(x + row + at_b[i]);
                    }
                    if (GRAD) {
                        ya[u][i].clear();
                        yb[u][i].clear();
                        if (h < h_end && has_a[i]) ya[u][i].load(dy + row + at_a[i]);
                        if (h < h_end && has_b[i]) yb[u][i].load(dy + row + at_b[i]);
                    }
                }
            }
            if (first) {  // (beneath the first loads)
                first = false;
                const uint64_t pos = static_cast<uint64_t>(position_of(p, token));
#pragma unroll
                for (int i = 0; i < R; ++i)
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const int k = INTERLEAVED ? at_a[i] / 2 + e : at_a[i] + e;
                        if (all_turned || (turned[i] && 2 * k < p.rot)) cos_sin<T>(pos * freq[i][e], p.factor, c[i][e], s[i][e]);
                        else c[i][e] = 1.0f, s[i][e] = 0.0f;
                        if (GRAD) s[i][e] = -s[i][e];  // back
                    }
            }
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) {
                const int h = hb + u * groups;
                if (hb - group + u * groups >= h_end) break;  // (the same for the whole warp)
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
                        if (all_turned || turned[i]) turn<V, INTERLEAVED>(c[i], s[i], ga[i], gb[i]);
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
                    float v, v1, g, g1;
                    unpack2(sum, v, v1);
                    unpack2(dot, g, g1);
                    v += v1;
                    g += g1;
                    for (int d = p.lanes / 2; d; d /= 2) {
                        v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
                        if (GRAD) g += __shfl_xor_sync(0xFFFFFFFFu, g, d);
                    }
                    v = rsqrtf(fmaf(v, inv_dim, p.eps));
                    scale = pack2(v, v);
                    if (GRAD) {
                        g = -(v * v * (g * inv_dim));
                        back = pack2(g, g);
                    }
                }
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    if (NORM) {
#pragma unroll
                        for (int e = 0; e < N; ++e) {
                            if (!GRAD) {
                                fa[i][e] = mul2(fa[i][e], mul2(scale, wa[i][e]));
                                fb[i][e] = mul2(fb[i][e], mul2(scale, wb[i][e]));
                            } else {
                                // (a head past the last has dz = x = 0)
                                dwa[i][e] = fma2(ga[i][e], mul2(fa[i][e], scale), dwa[i][e]);
                                dwb[i][e] = fma2(gb[i][e], mul2(fb[i][e], scale), dwb[i][e]);
                                ga[i][e] = mul2(scale, fma2(fa[i][e], back, mul2(ga[i][e], wa[i][e])));
                                gb[i][e] = mul2(scale, fma2(fb[i][e], back, mul2(gb[i][e], wb[i][e])));
                            }
                        }
                    }
                    if (!GRAD && (all_turned || turned[i])) turn<V, INTERLEAVED>(c[i], s[i], fa[i], fb[i]);
                    if (h < h_end) {
                        const int row = h * p.dim;
                        if (has_a[i]) Raw<T, V>::store(out + row + at_a[i], GRAD ? ga[i] : fa[i]);
                        if (has_b[i]) Raw<T, V>::store(out + row + at_b[i], GRAD ? gb[i] : fb[i]);
                    }
                }
            }
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
                for (int d = p.lanes; d < 32; d *= 2) {
                    va += __shfl_xor_sync(0xFFFFFFFFu, va, d);
                    vb += __shfl_xor_sync(0xFFFFFFFFu, vb, d);
                }
                if (group == 0 && has_a[i]) red[warp][at_a[i] + e] = va;
                if (group == 0 && has_b[i]) red[warp][at_b[i] + e] = vb;
            }
        __syncthreads();
        for (int d = threadIdx.x; d < p.dim; d += kRopeThreads) {
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < kRopeWarps; ++w) v += red[w][d];
            p.partial[static_cast<long long>(blockIdx.x) * p.dim + d] = v;
        }
    }
}

// dw = the sum of a side's partial rows, 32 columns a CTA.
__global__ void __launch_bounds__(1024) rope_sum_kernel(const __grid_constant__ RopeArgs p)
{
    __shared__ float red[32][33];
    grid_dep_wait();
    const RopeSide &sd = p.side[blockIdx.y];
    if (!sd.dw) return;
    const int x = threadIdx.x & 31, y = threadIdx.x / 32, col = blockIdx.x * 32 + x;
    const int first = blockIdx.y ? p.side[0].blocks * p.side[0].ctas : 0, n = sd.blocks * sd.ctas;
    float v = 0.0f;
    if (col < p.dim)
        for (int i = y; i < n; i += 32) v += p.partial[static_cast<long long>(first + i) * p.dim + col];
    red[y][x] = v;
    __syncthreads();
    v = red[x][y];
#pragma unroll
    for (int d = 16; d; d /= 2) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
    if (x == 0 && blockIdx.x * 32 + y < p.dim) sd.dw[blockIdx.x * 32 + y] = v;
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
    // a side's heads in one block where the tokens alone give every warp work: the angles are computed once a block
    a.block_heads = 32 / a.lanes * UNROLL;
    if (a.tokens >= kCtas * kRopeWarps / 2) a.block_heads = std::max({a.block_heads, a.side[0].heads, a.side[1].heads});
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
        if (a.pairs == a.lanes && a.dim == 2 * V * a.pairs)
            return a.interleaved ? launch_early(rope_kernel<T, V, UNROLL, GRAD, NORM, true, true>, grid, block, 0, s, a)
                                 : launch_early(rope_kernel<T, V, UNROLL, GRAD, NORM, false, true>, grid, block, 0, s, a);
    }
    return a.interleaved ? launch_early(rope_kernel<T, V, UNROLL, GRAD, NORM, true, false>, grid, block, 0, s, a)
                         : launch_early(rope_kernel<T, V, UNROLL, GRAD, NORM, false, false>, grid, block, 0, s, a);
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

// Rows of partial sums that launch_width may use, at most: a CTA a block of at
// least one head, or the share.
long long partial_rows(int heads, int kv_heads) { return kGradCtas + heads + kv_heads; }

struct RopeCall {
    long long tokens;
    int heads, kv_heads, dim, dtype, rot, interleaved, norm, index_bytes;
    float factor, eps;
    const float *inv_freq, *w_q, *w_k;
    const void *positions;
};

int check_call(const RopeCall &c)
{
    if (c.tokens < 0 || c.heads < 0 || c.kv_heads < 0 || c.heads + c.kv_heads < 1 || c.dim < 1 ||
        (c.dtype != CDG_F16 && c.dtype != CDG_BF16 && c.dtype != CDG_F32) || c.rot < 0 || c.rot > c.dim || c.rot % 2 ||
        (c.interleaved != 0 && c.interleaved != 1) || (c.norm != 0 && c.norm != 1) || (c.index_bytes != 4 && c.index_bytes != 8) ||
        !std::isfinite(c.factor) || !std::isfinite(c.eps) || c.eps < 0.0f || (c.rot > 0 && !c.inv_freq) ||
        (!c.norm && (c.w_q || c.w_k)))
        return CDG_ERR_INVALID_ARG;
    if (c.dim > kMaxHead || c.heads > kMaxHeads || c.kv_heads > kMaxHeads || c.tokens >= (1ll << 31)) return CDG_ERR_UNSUPPORTED;
    if (!aligned_to(c.inv_freq, 4) || !aligned_to(c.w_q, 4) || !aligned_to(c.w_k, 4) || !aligned_to(c.positions, c.index_bytes))
        return CDG_ERR_ALIGNMENT;
    return CDG_OK;
}

RopeArgs make_args(const RopeCall &c)
{
    RopeArgs a{};
    a.positions = c.positions;
    a.inv_freq = c.inv_freq;
    a.tokens = c.tokens;
    a.index_bytes = c.index_bytes;
    a.dim = c.dim;
    a.rot = c.rot;
    a.interleaved = c.interleaved;
    a.norm = c.norm;
    a.factor = c.factor;
    a.eps = c.eps;
    a.side[0].heads = c.heads;
    a.side[1].heads = c.kv_heads;
    a.side[0].w = c.w_q;
    a.side[1].w = c.w_k;
    return a;
}

int check_rows(const Rows &r)
{
    if (r.rows == 0 || r.width == 0) return CDG_OK;
    if (!r.p || r.ld < r.width) return CDG_ERR_INVALID_ARG;
    return aligned_to(r.p, r.esize) ? CDG_OK : CDG_ERR_ALIGNMENT;
}

// What a call reads beside its matrices.
struct SmallInputs {
    Extent e[4];
    SmallInputs(const RopeCall &c)
        : e{extent(c.inv_freq, c.rot / 2 * 4), extent(c.w_q, c.dim * 4), extent(c.w_k, c.dim * 4),
            extent(c.positions, static_cast<size_t>(c.tokens) * c.index_bytes)}
    {
    }
    bool meet(const Extent &x) const { return overlap(x, e[0]) || overlap(x, e[1]) || overlap(x, e[2]) || overlap(x, e[3]); }
};

bool same(const Rows &a, const Rows &b) { return a.p == b.p && a.ld == b.ld; }

}  // namespace
}  // namespace cdg

extern "C" {

int cdg_rope_frequencies(int rot, double base, double stretch, long long trained, double low, double high, float *inv_freq)
{
    if (rot < 0 || rot % 2 || rot > cdg::kMaxHead || !std::isfinite(base) || !(base > 0.0) || !std::isfinite(stretch) || !(stretch > 0.0) ||
        trained < 0 || (trained > 0 && !(low >= 0.0 && low < high && std::isfinite(high))) || (rot > 0 && !inv_freq))
        return CDG_ERR_INVALID_ARG;
    for (int i = 0; i < rot / 2; ++i) {
        const double f = std::pow(base, -2.0 * i / rot);
        double keep = 0.0;
        if (trained > 0) {
            const double turns = static_cast<double>(trained) * f / 6.283185307179586;
            keep = std::min(1.0, std::max(0.0, (turns - low) / (high - low)));
        }
        inv_freq[i] = static_cast<float>(f * (keep + (1.0 - keep) / stretch));
    }
    return CDG_OK;
}

int cdg_qk_rope(const void *q, long long ld_q, const void *k, long long ld_k, const void *positions, int index_bytes,
                long long tokens, int heads, int kv_heads, int dim, int dtype, const float *inv_freq, int rot, int interleaved,
                float factor, int norm, float eps, const float *w_q, const float *w_k, void *q_out, long long ld_qo, void *k_out,
                long long ld_ko, cdg_stream_t stream)
{
    using namespace cdg;
    const RopeCall c{tokens, heads, kv_heads, dim, dtype, rot, interleaved, norm, index_bytes, factor, eps, inv_freq, w_q, w_k, positions};
    int rc = check_call(c);
    if (rc != CDG_OK) return rc;
    const int es = dtype_bytes(dtype);
    const long long wq = static_cast<long long>(heads) * dim, wk = static_cast<long long>(kv_heads) * dim;
    const Rows in[2] = {{q, tokens, wq, ld_q, es}, {k, tokens, wk, ld_k, es}};
    const Rows out[2] = {{q_out, tokens, wq, ld_qo, es}, {k_out, tokens, wk, ld_ko, es}};
    for (const Rows &r : {in[0], in[1], out[0], out[1]})
        if ((rc = check_rows(r)) != CDG_OK) return rc;
    const SmallInputs small(c);
    for (int i = 0; i < 2; ++i) {
        if (out[i].width == 0) continue;
        if ((in[i].width && !same(out[i], in[i]) && overlap(out[i], in[i])) || (in[1 - i].width && overlap(out[i], in[1 - i])) ||
            small.meet(out[i].extent()))
            return CDG_ERR_ALIAS;
    }
    if (wq && wk && overlap(out[0], out[1])) return CDG_ERR_ALIAS;
    if (tokens == 0) return CDG_OK;
    RopeArgs a = make_args(c);
    for (int i = 0; i < 2; ++i) {
        a.side[i].x = in[i].p;
        a.side[i].ld_x = in[i].ld;
        a.side[i].out = const_cast<void *>(out[i].p);
        a.side[i].ld_out = out[i].ld;
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == CDG_F32   ? launch_rope<float, false>(a, s)
                          : dtype == CDG_F16 ? launch_rope<__half, false>(a, s)
                                             : launch_rope<__nv_bfloat16, false>(a, s);
    return e == cudaSuccess ? CDG_OK : CDG_ERR_CUDA;
}

size_t cdg_qk_rope_grad_workspace_bytes(long long tokens, int heads, int kv_heads, int dim)
{
    if (tokens < 0 || tokens >= (1ll << 31) || heads < 0 || kv_heads < 0 || heads > cdg::kMaxHeads || kv_heads > cdg::kMaxHeads || heads + kv_heads < 1 ||
        dim < 1 || dim > cdg::kMaxHead)
        return 0;
    return static_cast<size_t>(cdg::partial_rows(heads, kv_heads)) * dim * 4;
}

int cdg_qk_rope_grad(const void *q, long long ld_q, const void *k, long long ld_k, const void *positions, int index_bytes,
                     long long tokens, int heads, int kv_heads, int dim, int dtype, const float *inv_freq, int rot,
                     int interleaved, float factor, int norm, float eps, const float *w_q, const float *w_k, const void *dq_out,
                     long long ld_dqo, const void *dk_out, long long ld_dko, void *dq, long long ld_dq, void *dk, long long ld_dk,
                     float *dw_q, float *dw_k, void *workspace, cdg_stream_t stream)
{
    using namespace cdg;
    const RopeCall c{tokens, heads, kv_heads, dim, dtype, rot, interleaved, norm, index_bytes, factor, eps, inv_freq, w_q, w_k, positions};
    int rc = check_call(c);
    if (rc != CDG_OK) return rc;
    if ((!norm && (dw_q || dw_k)) || !workspace) return CDG_ERR_INVALID_ARG;
    const int es = dtype_bytes(dtype);
    const long long wq = static_cast<long long>(heads) * dim, wk = static_cast<long long>(kv_heads) * dim;
    // (without the norm the inputs are not read)
    const Rows x[2] = {{q, tokens, norm ? wq : 0, ld_q, es}, {k, tokens, norm ? wk : 0, ld_k, es}};
    const Rows dy[2] = {{dq_out, tokens, wq, ld_dqo, es}, {dk_out, tokens, wk, ld_dko, es}};
    const Rows dx[2] = {{dq, tokens, wq, ld_dq, es}, {dk, tokens, wk, ld_dk, es}};
    for (const Rows &r : {x[0], x[1], dy[0], dy[1], dx[0], dx[1]})
        if ((rc = check_rows(r)) != CDG_OK) return rc;
    if (!aligned_to(workspace, 16) || !aligned_to(dw_q, 4) || !aligned_to(dw_k, 4)) return CDG_ERR_ALIGNMENT;
    const SmallInputs small(c);
    const Extent ws = extent(workspace, cdg_qk_rope_grad_workspace_bytes(tokens, heads, kv_heads, dim)),
                 dw[2] = {extent(dw_q, dim * 4), extent(dw_k, dim * 4)};
    auto used = [](const Rows &r) { return r.rows > 0 && r.width > 0; };
    for (int i = 0; i < 2; ++i) {
        if (!used(dx[i])) continue;
        for (int j = 0; j < 2; ++j) {
            if (used(x[j]) && overlap(dx[i], x[j])) return CDG_ERR_ALIAS;
            if (used(dy[j]) && !(i == j && same(dx[i], dy[j])) && overlap(dx[i], dy[j])) return CDG_ERR_ALIAS;
        }
    }
    if (used(dx[0]) && used(dx[1]) && overlap(dx[0], dx[1])) return CDG_ERR_ALIAS;
    for (const Rows &r : {x[0], x[1], dy[0], dy[1], dx[0], dx[1]}) {
        if (!used(r)) continue;
        const Extent e = r.extent();
        if (overlap(e, ws) || overlap(e, dw[0]) || overlap(e, dw[1])) return CDG_ERR_ALIAS;
        if ((r.p == dq || r.p == dk) && small.meet(e)) return CDG_ERR_ALIAS;
    }
    if (small.meet(ws) || small.meet(dw[0]) || small.meet(dw[1]) || overlap(ws, dw[0]) || overlap(ws, dw[1]) || overlap(dw[0], dw[1]))
        return CDG_ERR_ALIAS;
    RopeArgs a = make_args(c);
    for (int i = 0; i < 2; ++i) {
        a.side[i].x = x[i].p;
        a.side[i].ld_x = x[i].ld;
        a.side[i].dy = dy[i].p;
        a.side[i].ld_dy = dy[i].ld;
        a.side[i].out = const_cast<void *>(dx[i].p);
        a.side[i].ld_out = dx[i].ld;
    }
    a.side[0].dw = dw_q;
    a.side[1].dw = dw_k;
    a.partial = static_cast<float *>(workspace);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    if (tokens > 0)
        e = dtype == CDG_F32   ? launch_rope<float, true>(a, s)
            : dtype == CDG_F16 ? launch_rope<__half, true>(a, s)
                               : launch_rope<__nv_bfloat16, true>(a, s);
    if (e == cudaSuccess && (dw_q || dw_k)) e = launch_early(rope_sum_kernel, dim3((dim + 31) / 32, 2), dim3(1024), 0, s, a);
    return e == cudaSuccess ? CDG_OK : CDG_ERR_CUDA;
}

}  // extern "C"
