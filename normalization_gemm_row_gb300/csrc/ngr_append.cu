// ngr_append.cu -- new tokens' keys and values into a paged cache, keys and
// queries rotated by their position on the way.
//
//   angle(t, i) = positions[t] inv_freq[i],  i < rot / 2
//   (a, b) -> (a cos - b sin, a sin + b cos) for the pairs (i, i + rot / 2),
//   or (2i, 2i + 1) interleaved; dimensions from rot on are copied.
//
// Every element is read once and written once, so memory bounds it: 2 (H + 2 G)
// D elements a token.  A thread moves one pair of 16-byte pieces (a unit),
// whose loads start before the position and the page are known, so that
// a block waits for memory twice (position, table) and not three times.
#include "ngr.h"
#include "ngr_entry.h"
#include "ngr_internal.h"
#include "ngr_kv.h"
#include "ngr_mma.cuh"

namespace ngr {

namespace {

// f / (2 pi) modulo 1 as a 64-bit fraction: the 24-bit significand times the
// first 128 bits of 1 / (2 pi), shifted by f's exponent.  A position times
// this, modulo 2^64, is the angle in turns to 2^-64 of a turn per position:
// the product position x f in FP32 would be 2^-7 off at position 2^17, and
// FP64 has a sixty-fourth of FP32's rate here.  (0 from 2^88 on.)
__device__ __forceinline__ unsigned long long turn_fraction(float f)
{
    constexpr unsigned long long kHi = 0x28be60db9391054aull, kLo = 0x7f09d5f47d4d3770ull;
    const uint32_t bits = __float_as_uint(f);
    const int e = static_cast<int>((bits >> 23) & 255u);
    const unsigned long long m = (bits & 0x7FFFFFu) | (e ? 0x800000u : 0u);
    const int r = 64 - ((e ? e : 1) - 150);
    const unsigned long long p0 = m * kLo, c = __umul64hi(m, kLo), mid = m * kHi, p1 = mid + c,
                             p2 = __umul64hi(m, kHi) + (p1 < mid ? 1u : 0u);
    unsigned long long lo = 0, hi = 0;      // the words that the shift by r leaves, before its last r % 64 bits
    if (r >= 0) {
        const int w = r >> 6;
        lo = w == 0 ? p0 : w == 1 ? p1 : w == 2 ? p2 : 0;
        hi = w == 0 ? p1 : w == 1 ? p2 : 0;
    }
    const int b = r & 63;
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

template <bool BF16>
__device__ __forceinline__ float to_f(uint16_t v)
{
    if (BF16) return __uint_as_float(static_cast<uint32_t>(v) << 16);
    return __half2float(__ushort_as_half(v));
}
template <bool BF16>
__device__ __forceinline__ uint16_t from_f(float v)
{
    return static_cast<uint16_t>(pack16<BF16>(v, 0.0f));
}

// The units of a head: of each, two pieces of VEC elements from `first` and
// `second` on (second < 0: one piece).  Pair units rotate the pieces against
// one another, inner units each within itself; others are copied.
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

template <bool BF16, int VEC, bool INTERLEAVED>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const __grid_constant__ AppendArgs a)
{
    using P = typename Piece<VEC>::T;
    union Data {
        P p;
        uint16_t e[VEC];
    };
    __shared__ float2 turn[kAttendMaxDim / 2];
    if (a.err && blockIdx.x == 0) {
        // The error word by one block: the others leave bad tokens out, and
        // without a launch of its own nothing could clear the word for them.
        bool bad = false;
        for (int t = threadIdx.x; t < a.T; t += kAppendThreads) page_of(a, t, a.positions[t], &bad);
        if (__syncthreads_or(bad) == 0) {
            if (threadIdx.x == 0) *a.err = 0;
        } else if (threadIdx.x == 0) {
            *a.err = kDevErrPage;
        }
        return;
    }
    const unsigned block = blockIdx.x - (a.err ? 1u : 0u);
    const int t = static_cast<int>(block / static_cast<unsigned>(a.blocks_per_token));
    const int part = static_cast<int>(block - static_cast<unsigned>(t) * a.blocks_per_token);
    const int position = a.positions[t];

    int i = part * kAppendThreads + static_cast<int>(threadIdx.x);
    const int per = units_of_head(VEC, INTERLEAVED, a.D, a.rot), turned = (a.H + a.G) * per;
    const bool any_turned = part * kAppendThreads < turned;
    const uint16_t *src = nullptr;
    int head = 0, what = 3;     // 0 q, 1 k, 2 v, 3 nothing
    Unit u = {0, -1, kCopy};
    if (i < turned) {
        head = i / per;
        u = unit_of<VEC, INTERLEAVED>(i - head * per, a.D, a.rot);
        what = head < a.H ? 0 : 1;
        if (what == 0) {
            src = static_cast<const uint16_t *>(a.q) + t * a.q_token + head * a.q_head;
        } else {
            head -= a.H;
            src = static_cast<const uint16_t *>(a.k) + t * a.k_token + head * a.k_head;
        }
    } else {
        i -= turned;
        const int each = units_of_head(VEC, false, a.D, 0);
        if (i < a.G * each) {
            head = i / each;
            u = unit_of<VEC, false>(i - head * each, a.D, 0);
            what = 2;
            src = static_cast<const uint16_t *>(a.v) + t * a.v_token + head * a.v_head;
        }
    }
    Data x, y;
    if (src) {
        x.p = *reinterpret_cast<const P *>(src + u.first);
        if (u.second >= 0) y.p = *reinterpret_cast<const P *>(src + u.second);
    }
    bool bad = false;
    const int page = page_of(a, t, position, &bad);
    if (page < 0) return;      // (the whole block: it has one token)
    if (any_turned) {
        for (int f = threadIdx.x; f < a.rot / 2; f += kAppendThreads) turn[f] = rotation(a.inv_freq[f], position);
        __syncthreads();
    }
    if (!src) return;
    if (u.kind == kPair) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float2 cs = turn[INTERLEAVED ? u.first / 2 : u.first + e];
            const float p = to_f<BF16>(x.e[e]), q = to_f<BF16>(y.e[e]);
            x.e[e] = from_f<BF16>(p * cs.x - q * cs.y);
            y.e[e] = from_f<BF16>(p * cs.y + q * cs.x);
        }
    } else if (INTERLEAVED && VEC > 1 && u.kind == kInner) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            Data &d = h ? y : x;
            const int at = h ? u.second : u.first;
            if (at < 0 || at >= a.rot) continue;
#pragma unroll
            for (int e = 0; e + 1 < VEC; e += 2) {
                const float2 cs = turn[(at + e) / 2];
                const float p = to_f<BF16>(d.e[e]), q = to_f<BF16>(d.e[e + 1]);
                d.e[e] = from_f<BF16>(p * cs.x - q * cs.y);
                d.e[e + 1] = from_f<BF16>(p * cs.y + q * cs.x);
            }
        }
    }
    uint16_t *dst;
    if (what == 0) {
        dst = static_cast<uint16_t *>(a.q_out) + t * a.qo_token + head * a.qo_head;
    } else {
        const int64_t slot = position - position / a.kv.page_size * a.kv.page_size;
        dst = what == 1 ? static_cast<uint16_t *>(a.kv.k) + page * a.kv.k_page + slot * a.kv.k_token + head * a.kv.k_head
                        : static_cast<uint16_t *>(a.kv.v) + page * a.kv.v_page + slot * a.kv.v_token + head * a.kv.v_head;
    }
    *reinterpret_cast<P *>(dst + u.first) = x.p;
    if (u.second >= 0) *reinterpret_cast<P *>(dst + u.second) = y.p;
}

template <bool BF16, int VEC>
void launch(bool interleaved, const AppendArgs &a, unsigned grid, cudaStream_t stream)
{
    if (interleaved)
        append_kernel<BF16, VEC, true><<<grid, kAppendThreads, 0, stream>>>(a);
    else
        append_kernel<BF16, VEC, false><<<grid, kAppendThreads, 0, stream>>>(a);
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

int64_t append_units(int vec, bool interleaved, int64_t H, int64_t G, int64_t D, int64_t rot)
{
    const int d = static_cast<int>(D), r = static_cast<int>(rot);
    return (H + G) * units_of_head(vec, interleaved, d, r) + G * units_of_head(vec, false, d, 0);
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
