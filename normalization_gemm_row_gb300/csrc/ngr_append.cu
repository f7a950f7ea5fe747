// ngr_append.cu -- new tokens' keys and values into a paged cache, keys and
// queries rotated by their position on the way.
//
//   angle(t, i) = positions[t] inv_freq[i],  i < rot / 2
//   (a, b) -> (a cos - b sin, a sin + b cos) for the pairs (i, i + rot / 2),
//   or (2i, 2i + 1) interleaved; dimensions from rot on are copied.
//
// Every element is read once and written once, so memory bounds it: 2 (H + 2 G)
// D elements a token.  A thread moves pairs of 16-byte pieces (units), whose
// loads start before the position and the page are known, so that a block
// waits for memory twice (position, table) and not three times.  8192 tokens
// of 64 + 2 x 8 heads of 128: 62 to 64 us, 5.3 TB/s, in interleaved pairs or
// half rotated as well; one token: 5 to 6 us.
#include "ngr.h"
#include "ngr_entry.h"
#include "ngr_internal.h"
#include "ngr_kv.h"
#include "ngr_mma.cuh"

namespace ngr {

namespace {

// f / (2 pi) modulo 1 as a 64-bit fraction: the 24-bit significand times the
// first 192 bits of 1 / (2 pi), shifted by f's exponent, which is at most 104.
// Off by less than 2^-62, for any finite f.  A position times this, modulo
// 2^64, is the angle in turns: the product position x f in FP32 would be 2^-7
// off at position 2^17, and FP64 has a sixty-fourth of FP32's rate here.
__device__ __forceinline__ unsigned long long turn_fraction(float f)
{
    constexpr unsigned long long k2 = 0x28be60db9391054aull, k1 = 0x7f09d5f47d4d3770ull, k0 = 0x36d8a5664f10e410ull;
    const uint32_t bits = __float_as_uint(f);
    const int e = static_cast<int>((bits >> 23) & 255u);
    const unsigned long long m = (bits & 0x7FFFFFu) | (e ? 0x800000u : 0u);
    const int r = 128 - ((e ? e : 1) - 150);      // 24 and more, for finite f
    // the product's words: its shift by r leaves those from number r / 64 on
    unsigned long long p[6] = {m * k0, 0, 0, 0, 0, 0};
    const unsigned long long mid1 = m * k1, mid2 = m * k2;
    p[1] = mid1 + __umul64hi(m, k0);
    p[2] = mid2 + __umul64hi(m, k1) + (p[1] < mid1 ? 1u : 0u);
    p[3] = __umul64hi(m, k2) + (p[2] < mid2 ? 1u : 0u);
    const int w = r >> 6, b = r & 63;
    unsigned long long lo = 0, hi = 0;
#pragma unroll
    for (int i = 0; i < 5; ++i)
        if (i == w) {
            lo = p[i];
            hi = p[i + 1];
        }
    const unsigned long long u = (lo >> b) | (b ? hi << (64 - b) : 0);
    return bits >> 31 ? 0 - u : u;
}

// (cos, sin) of position x f.
__device__ __forceinline__ float2 rotation(float f, int position)
{
    const long long turns = static_cast<long long>(turn_fraction(f) * static_cast<unsigned long long>(position));
    float s, c;
    sincospif(static_cast<float>(turns) * 1.0842021724855044e-19f, &s, &c);   // 2^-63: half turns
    return fabsf(f) < INFINITY ? make_float2(c, s) : make_float2(NAN, NAN);
}

template <int VEC> struct Piece;
template <> struct Piece<8> { using T = uint4; };
template <> struct Piece<4> { using T = uint2; };
template <> struct Piece<2> { using T = uint32_t; };
template <> struct Piece<1> { using T = uint16_t; };

// Two elements of a piece (or its only one) as floats, and back.
template <bool BF16, int VEC>
__device__ __forceinline__ float2 get2(const uint16_t (&e)[VEC], int i)
{
    return unpack16<BF16>(VEC > 1 ? reinterpret_cast<const uint32_t *>(e)[i / 2] : static_cast<uint32_t>(e[0]));
}
template <bool BF16, int VEC>
__device__ __forceinline__ void set2(uint16_t (&e)[VEC], int i, float x, float y)
{
    const uint32_t v = pack16<BF16>(x, y);
    if (VEC > 1) reinterpret_cast<uint32_t *>(e)[i / 2] = v;
    else e[0] = static_cast<uint16_t>(v);
}

// The units of a head: of each, two pieces of VEC elements from `first` and
// `second` on (second < 0: one piece; first past D: none).  Pair units rotate
// the pieces against one another, inner units each within itself; others are
// copied.
enum { kCopy = 0, kPair = 1, kInner = 2 };
struct Unit {
    int first, second, kind;
};
template <int VEC, bool INTERLEAVED>
__device__ __forceinline__ Unit unit_of(int i, int D, int rot)
{
    Unit u;
    if (INTERLEAVED && VEC > 1) {
        u.first = 2 * i * VEC;
        u.second = u.first + VEC;
        u.kind = kInner;
    } else {
        const int pairs = rot / 2 / VEC;
        if (i < pairs) {
            u.first = INTERLEAVED ? 2 * i : i * VEC;
            u.second = INTERLEAVED ? 2 * i + 1 : rot / 2 + i * VEC;
            u.kind = kPair;
            return u;
        }
        u.first = rot + 2 * (i - pairs) * VEC;
        u.second = u.first + VEC;
        u.kind = kCopy;
    }
    if (u.second >= D) u.second = -1;
    return u;
}
__host__ __device__ constexpr int units_of_head(int vec, bool interleaved, int D, int rot)
{
    const int pairs = interleaved && vec > 1 ? 0 : rot / 2 / vec, rest = interleaved && vec > 1 ? D : D - rot;
    return pairs + (rest + 2 * vec - 1) / (2 * vec);
}

// The token's slot in the cache: its page, or -1 if the token takes none (a
// negative position) or has none (*bad).
__device__ __forceinline__ int page_of(const AppendArgs &a, int t, int position, bool *bad)
{
    if (position < 0) return -1;
    const int row = a.rows ? a.rows[t] : t;
    int page = -1;
    if (row >= 0 && row < a.kv.rows && position < a.kv.capacity)
        page = a.kv.table[row * a.kv.table_stride + position / a.kv.page_size];
    if (page < 0 || page >= a.kv.pages) {
        *bad = true;
        page = -1;
    }
    return page;
}

// A block has one token: its threads stand for `a.units` units of
// threads / a.units heads, EACH times over, so that a thread's units are the
// same one of different heads and turn by the same angles.
template <bool BF16, int VEC, bool INTERLEAVED, int EACH>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const __grid_constant__ AppendArgs a)
{
    using P = typename Piece<VEC>::T;
    union Data {
        P p;
        uint16_t e[VEC];
        __device__ Data() {}
    };
    constexpr int kAngles = INTERLEAVED && VEC > 1 ? VEC / 2 : VEC;     // of a piece
    __shared__ float2 turn[kAttendMaxDim / 2];
    const int threads = static_cast<int>(blockDim.x);
    if (a.err && blockIdx.x == 0) {
        // The error word by one block: the others leave bad tokens out, and
        // without a launch of its own nothing could clear the word for them.
        // It goes over all tokens, as many at once as it has threads, and is
        // the longest block where those are few: 8192 tokens of 3 heads of 64
        // 296 us (10 without a workspace), of 48 heads of 64 92 (22), of 80
        // heads of 128 62 (62).
        bool bad = false;
        for (int t = threadIdx.x; t < a.T; t += threads) page_of(a, t, a.positions[t], &bad);
        const int any = __syncthreads_or(bad);
        if (threadIdx.x == 0) *a.err = any ? kDevErrPage : 0;
        return;
    }
    const unsigned block = blockIdx.x - (a.err ? 1u : 0u);
    const int t = static_cast<int>(block / static_cast<unsigned>(a.blocks_per_token));
    const int part = static_cast<int>(block - static_cast<unsigned>(t) * a.blocks_per_token);
    const int position = a.positions[t];

    const int step = threads / a.units, row = static_cast<int>(threadIdx.x) / a.units;
    const int i = static_cast<int>(threadIdx.x) - row * a.units, first = part * step * EACH + row;
    const Unit turned = unit_of<VEC, INTERLEAVED>(i, a.D, a.rot), plain = unit_of<VEC, false>(i, a.D, 0);
    Data x[EACH], y[EACH];
#pragma unroll
    for (int n = 0; n < EACH; ++n) {
        const int head = first + n * step;
        const uint16_t *src;
        if (head < a.H) src = static_cast<const uint16_t *>(a.q) + t * a.q_token + head * a.q_head;
        else if (head < a.H + a.G) src = static_cast<const uint16_t *>(a.k) + t * a.k_token + (head - a.H) * a.k_head;
        else if (head < a.H + 2 * a.G) src = static_cast<const uint16_t *>(a.v) + t * a.v_token + (head - a.H - a.G) * a.v_head;
        else continue;
        const Unit &u = head < a.H + a.G ? turned : plain;
        if (u.first < a.D) x[n].p = *reinterpret_cast<const P *>(src + u.first);
        if (u.second >= 0) y[n].p = *reinterpret_cast<const P *>(src + u.second);
    }
    bool bad = false;
    const int page = page_of(a, t, position, &bad);
    if (page < 0) return;      // (the whole block: it has one token)
    for (int f = threadIdx.x; f < a.rot / 2; f += threads) turn[f] = rotation(a.inv_freq[f], position);
    __syncthreads();
    // the angles of the pieces, one after the other in `turn`
    constexpr int kTurned = INTERLEAVED && VEC > 1 ? 2 : 1;     // pieces that have angles of their own
    float2 cs[kTurned][kAngles];
    bool turns[kTurned];
#pragma unroll
    for (int h = 0; h < kTurned; ++h) {
        const int at = h ? turned.second : turned.first;
        turns[h] = turned.kind == kInner ? at >= 0 && at < a.rot : turned.kind == kPair;
        const int from = turned.kind == kInner || INTERLEAVED ? at / 2 : at;
#pragma unroll
        for (int e = 0; e < kAngles; ++e) cs[h][e] = turns[h] ? turn[from + e] : make_float2(1.0f, 0.0f);
    }
    const int64_t slot = position - position / a.kv.page_size * a.kv.page_size;
#pragma unroll
    for (int n = 0; n < EACH; ++n) {
        const int head = first + n * step;
        uint16_t *dst;
        if (head < a.H)
            dst = static_cast<uint16_t *>(a.q_out) + t * a.qo_token + head * a.qo_head;
        else if (head < a.H + a.G)
            dst = static_cast<uint16_t *>(a.kv.k) + page * a.kv.k_page + slot * a.kv.k_token + (head - a.H) * a.kv.k_head;
        else if (head < a.H + 2 * a.G)
            dst = static_cast<uint16_t *>(a.kv.v) + page * a.kv.v_page + slot * a.kv.v_token + (head - a.H - a.G) * a.kv.v_head;
        else
            break;
        const bool is_v = head >= a.H + a.G;
        if (!is_v) {
            if constexpr (INTERLEAVED && VEC > 1) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (!turns[h]) continue;
                    Data &d = h ? y[n] : x[n];
#pragma unroll
                    for (int e = 0; e < VEC; e += 2) {
                        const float2 v = get2<BF16>(d.e, e), c = cs[h][e / 2];
                        set2<BF16>(d.e, e, v.x * c.x - v.y * c.y, v.x * c.y + v.y * c.x);
                    }
                }
            } else if (turns[0]) {
#pragma unroll
                for (int e = 0; e < VEC; e += 2) {
                    const float2 p = get2<BF16>(x[n].e, e), q = get2<BF16>(y[n].e, e);
                    const float2 c = cs[0][e], d = cs[0][VEC > 1 ? e + 1 : e];
                    set2<BF16>(x[n].e, e, p.x * c.x - q.x * c.y, p.y * d.x - q.y * d.y);
                    set2<BF16>(y[n].e, e, p.x * c.y + q.x * c.x, p.y * d.y + q.y * d.x);
                }
            }
        }
        const Unit &u = is_v ? plain : turned;
        if (u.first < a.D) *reinterpret_cast<P *>(dst + u.first) = x[n].p;
        if (u.second >= 0) *reinterpret_cast<P *>(dst + u.second) = y[n].p;
    }
}

template <bool BF16, int VEC>
void launch(bool interleaved, const AppendArgs &a, unsigned grid, cudaStream_t stream)
{
    const unsigned threads = static_cast<unsigned>(a.threads);
    if (a.each > 1) {
        if (interleaved) append_kernel<BF16, VEC, true, kAppendEach><<<grid, threads, 0, stream>>>(a);
        else append_kernel<BF16, VEC, false, kAppendEach><<<grid, threads, 0, stream>>>(a);
    } else {
        if (interleaved) append_kernel<BF16, VEC, true, 1><<<grid, threads, 0, stream>>>(a);
        else append_kernel<BF16, VEC, false, 1><<<grid, threads, 0, stream>>>(a);
    }
}
template <bool BF16>
void launch(int vec, bool interleaved, const AppendArgs &a, unsigned grid, cudaStream_t stream)
{
    if (vec == 8) launch<BF16, 8>(interleaved, a, grid, stream);
    else if (vec == 4) launch<BF16, 4>(interleaved, a, grid, stream);
    else if (vec == 2) launch<BF16, 2>(interleaved, a, grid, stream);
    else launch<BF16, 1>(interleaved, a, grid, stream);
}

}  // namespace

int append_units(int vec, bool interleaved, int64_t D, int64_t rot)
{
    const int d = static_cast<int>(D), turned = units_of_head(vec, interleaved, d, static_cast<int>(rot));
    const int plain = units_of_head(vec, false, d, 0);
    return turned > plain ? turned : plain;
}

int launch_append(bool bf16, int vec, bool interleaved, const AppendArgs &a, cudaStream_t stream)
{
    const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(a.T) * a.blocks_per_token) + (a.err ? 1u : 0u);
    if (bf16) launch<true>(vec, interleaved, a, grid, stream);
    else launch<false>(vec, interleaved, a, grid, stream);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? 0 : record_cuda_error("rotated append launch", e, cudaGetErrorString(e));
}

}  // namespace ngr
