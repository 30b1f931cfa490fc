// k_block8.cuh -- block-scaled E4M3 matrices: writing, reading back, products.
//
// A block8 matrix holds rows of d values as E4M3 codes with one power-of-two scale
// per block of 128 values along the row. With a the largest magnitude among a
// block's finite values, its exponent is
//     e = the smallest integer with a <= 448 * 2^e, within [-117, 119]   (0 if a = 0)
// and a value x is held as c = e4m3(x * 2^-e), nearest even, standing for c * 2^e.
// The scaling is exact, so each value is rounded once; codes are floating point, so
// a power of two costs them no relative accuracy (only up to one bit of the range
// below the block's maximum). Four significant bits and a smallest value of
// 2^-9 * 2^-117 = 2^-126 make every held value exact in fp32 and in bf16, and the
// largest, 448 * 2^119 = 1.75 * 2^127, is finite there (fp32 values beyond it
// saturate). NaN and infinities are held as NaN and leave their block's scale alone.
//
// Layout: codes are rows of round_up(d, 16) bytes (TMA wants 16-byte rows), zeros
// past d. Exponents are bytes e + 127 (E8M0) in the order in which the tensor cores
// take scale factors, so that a product copies them to tensor memory as they are:
// [row / 128][block / 4][row % 32][(row / 32) % 4][block % 4], 512 bytes for each
// 128 rows x 4 blocks (block8_scale_at).
#pragma once

#include "k_assign.cuh"
#include "k_data.cuh"
#include "ring.cuh"

namespace em {
namespace b8 {

constexpr int kBlock = 128;       // values per scale
constexpr int kMinExp = -117, kMaxExp = 119;
constexpr int kAtomBytes = 512;   // exponents of 128 rows x 4 blocks

__host__ __device__ __forceinline__ int64_t scale_at(int64_t row, int64_t block, int64_t groups) {
    return ((((row >> 7) * groups + (block >> 2)) * 32 + (row & 31)) * 4 + ((row >> 5) & 3)) * 4 + (block & 3);
}

// The exponent of a block from the bit pattern of its largest finite magnitude:
// 448 = 1.75 * 2^8, so e is the magnitude's own exponent less 8, one more where its
// mantissa is above 1.75.
__device__ __forceinline__ int block_exponent(uint32_t amax_bits) {
    const int e = (int)(amax_bits >> 23) - 135 + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return amax_bits == 0u ? 0 : min(max(e, kMinExp), kMaxExp);
}

// NaN for NaN and infinities, x otherwise.
__device__ __forceinline__ float finite_or_nan(float x) {
    return (__float_as_uint(x) & 0x7F800000u) == 0x7F800000u ? __int_as_float(0x7FC00000) : x;
}

// Codes of 4 scaled values (the first in the low byte). Infinities must have been made
// NaN before: the conversion would saturate them.
__device__ __forceinline__ uint32_t encode4(const float v[4], float inverse) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(v[1] * inverse), "f"(v[0] * inverse));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(v[3] * inverse), "f"(v[2] * inverse));
    return (uint32_t)lo | ((uint32_t)hi << 16);
}

__device__ __forceinline__ void decode4(uint32_t codes, float v[4]) {
    uint32_t h0, h1;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h0) : "h"((uint16_t)(codes & 0xFFFFu)));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h1) : "h"((uint16_t)(codes >> 16)));
    __half2 a, b;
    memcpy(&a, &h0, 4);
    memcpy(&b, &h1, 4);
    const float2 fa = __half22float2(a), fb = __half22float2(b);
    v[0] = fa.x; v[1] = fa.y; v[2] = fb.x; v[3] = fb.y;
}

// 2^e of an exponent byte as a float (bytes 10..246 are written; 0 would be a
// subnormal and reads as 0).
__device__ __forceinline__ float scale_of(uint8_t byte) { return __uint_as_float((uint32_t)byte << 23); }

template <class T> __device__ __forceinline__ float to_f32(T v);
template <> __device__ __forceinline__ float to_f32(float v) { return v; }
template <> __device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <> __device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <class T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f32(float v) { return __float2half_rn(v); }

template <class T, int N>
struct alignas(N * sizeof(T)) Vec { T v[N]; };

// The widest access, in elements, that rows at `base` with `ld` elements between them
// allow: 16 bytes, 8 bytes, or single elements.
template <class T>
__host__ __device__ __forceinline__ int vector_width(const void* base, int64_t ld) {
    for (int w = 16 / (int)sizeof(T); w >= 8 / (int)sizeof(T); w >>= 1)
        if (reinterpret_cast<uintptr_t>(base) % (w * sizeof(T)) == 0 && ld % w == 0) return w;
    return 1;
}

template <class T, int W>
__device__ __forceinline__ void store8_as(T* p, const float v[8]) {
#pragma unroll
    for (int q = 0; q < 8 / W; ++q) {
        Vec<T, W> x;
#pragma unroll
        for (int t = 0; t < W; ++t) x.v[t] = from_f32<T>(v[q * W + t]);
        reinterpret_cast<Vec<T, W>*>(p)[q] = x;
    }
}

template <class T>
__device__ __forceinline__ void store8(T* p, int left, int width, const float v[8]) {
    if (left >= 8 && width == 16 / (int)sizeof(T)) {
        store8_as<T, 16 / sizeof(T)>(p, v);
    } else if (left >= 8 && width > 1) {
        store8_as<T, 8 / sizeof(T)>(p, v);
    } else {
#pragma unroll
        for (int t = 0; t < 8; ++t)
            if (t < left) p[t] = from_f32<T>(v[t]);
    }
}

// Division of 32-bit numbers by a fixed one, exact for every dividend below 2^31
// (Granlund and Montgomery, "Division by invariant integers using multiplication",
// PLDI 1994: with l = ceil(log2 div), m = floor(2^(31 + l) / div) + 1 has a relative
// error of at most 2^-31 in the quotient's direction).
struct FastDiv {
    uint32_t div = 1;
    uint64_t mul = 1ull << 31;
    int shift = 31;
    explicit FastDiv(uint32_t d) : div(d) {
        int l = 0;
        while ((1ull << l) < d) ++l;
        shift = 31 + l;
        mul = (1ull << shift) / d + 1;
    }
    __host__ __device__ __forceinline__ uint32_t quotient(uint32_t x) const { return (uint32_t)((x * mul) >> shift); }
};

// Where row i of a call goes (write) or comes from (read): row first + i, or slots[i].
// Returns -1 for a row to leave out: slot -1 (padding), or a slot outside the matrix,
// which also raises EM_E_BOUNDS.
__device__ __forceinline__ int64_t slot_of(const int64_t* __restrict__ slots, int64_t first, int64_t i, int64_t rows,
                                           int* status) {
    if (!slots) return first + i;
    const int64_t s = slots[i];
    if (s >= 0 && s < rows) return s;
    if (s != -1) raise_error(status, EM_E_BOUNDS);
    return -1;
}

// Several rows of one call may name the same slot: the last of them stays, whole.
// Calls of up to kScanRows rows look for a later row with the same slot where they
// write; longer calls run this pass first, which leaves in claims[slot] the last row
// of this call that names it. Whoever takes a later row's place there puts it back: an
// entry that this call did not make (its row does not name the slot) is no row of this
// call, so the array needs no initial value, and a captured call can be replayed at any
// time. The loop ends, since what it puts back grows.
// The pass costs a second launch, the scan grows with the rows. Of 768 bf16 values each,
// in a captured graph: 32 rows 2.5 us with the scan and 3.4 with the pass, 128 3.3 and 3.6,
// 512 5.8 and 3.6, 1,024 9.5 and 3.7; called one by one, where the host's part of the
// second launch counts, 512 rows 6.2 and 8.3.
constexpr int kScanRows = 512;

__global__ void k_block8_claim(const int64_t* __restrict__ slots, int64_t n, int64_t rows, int* __restrict__ claims) {
    pdl_wait();
    pdl_release();
    for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t s = slots[i];
        if (s < 0 || s >= rows) continue;
        for (int mine = (int)i;;) {
            const int old = atomicExch(claims + s, mine);
            if (old <= mine || old >= n || slots[old] != s) break;
            mine = old;
        }
    }
}

// Whether row i is the one that stays in its slot s. `lanes` (8, 16 or 32) neighbouring
// lanes ask for the same row, `lane` is this one's place among them; all lanes of the
// warp call it together.
__device__ __forceinline__ bool last_of_slot(const int64_t* __restrict__ slots, const int* __restrict__ claims,
                                             int64_t i, int64_t n, int64_t s, int lane, int lanes) {
    if (claims) return s < 0 || claims[s] == (int)i;
    bool later = false;
    if (s >= 0)
        for (int64_t j = i + 1 + lane; j < n; j += lanes) later |= slots[j] == s;
    const uint32_t all = __ballot_sync(0xFFFFFFFFu, later);
    const int shift = threadIdx.x & 31 & ~(lanes - 1);
    return ((all >> shift) & (0xFFFFFFFFu >> (32 - lanes))) == 0u;
}

// Words of magnitudes: the larger of each part; NaN gives way.
template <class T> __device__ __forceinline__ uint32_t max_parts(uint32_t a, uint32_t b);
template <> __device__ __forceinline__ uint32_t max_parts<float>(uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
}
template <> __device__ __forceinline__ uint32_t max_parts<__nv_bfloat16>(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
template <> __device__ __forceinline__ uint32_t max_parts<__half>(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Part s of a word as fp32, and an fp32 value put in its place.
template <class T>
__device__ __forceinline__ float part_of(uint32_t w, int s) {
    if (sizeof(T) == 4) return __uint_as_float(w);
    const uint16_t h = (uint16_t)(w >> (16 * s));
    T v;
    memcpy(&v, &h, sizeof(T) < 2 ? sizeof(T) : 2);
    return to_f32(v);
}
template <class T>
__device__ __forceinline__ uint32_t with_part(uint32_t w, int s, float f) {
    if (sizeof(T) == 4) return __float_as_uint(f);
    const T v = from_f32<T>(f);
    uint16_t h;
    memcpy(&h, &v, 2);
    return s ? (w & 0xFFFFu) | ((uint32_t)h << 16) : (w & 0xFFFF0000u) | h;
}

// The work of the row kernels: (row, block) pairs in row order, 16 lanes per pair with
// 8 consecutive values each, two pairs per warp and step, kSteps steps in flight.
// Short rows fill a warp as well as long ones (a row of 96 values is one pair).
constexpr int kSteps = 4;
constexpr int kPairsPerWarp = 2 * kSteps;

// The (row, block) pairs of a lane: first the pair `f`, then every second one.
struct Pairs {
    int row[kSteps], b[kSteps];
    __device__ __forceinline__ Pairs(uint32_t f, const FastDiv& nb) {
        const int nbi = (int)nb.div;
        row[0] = (int)nb.quotient(f);
        b[0] = (int)f - row[0] * nbi;
#pragma unroll
        for (int s = 1; s < kSteps; ++s) {  // one row on at most, or two where a row is one block
            b[s] = b[s - 1] + 2;
            row[s] = row[s - 1];
#pragma unroll
            for (int q = 0; q < 2; ++q)
                if (b[s] >= nbi) {
                    b[s] -= nbi;
                    ++row[s];
                }
        }
    }
};

// N values of type T as words.
template <class T, int N>
struct Values {
    static constexpr int kWords = N * (int)sizeof(T) / 4, PW = 4 / (int)sizeof(T);
    static constexpr uint32_t kAbs = sizeof(T) == 4 ? 0x7FFFFFFFu : 0x7FFF7FFFu;
    uint32_t w[kWords];
    __device__ __forceinline__ void load16(const T* p) {  // 16-byte aligned
#pragma unroll
        for (int q = 0; q < kWords; q += 4) {
            const uint4 u = reinterpret_cast<const uint4*>(p)[q / 4];
            w[q] = u.x; w[q + 1] = u.y; w[q + 2] = u.z; w[q + 3] = u.w;
        }
    }
    __device__ __forceinline__ void load32(const T* p) {  // 32-byte aligned
#pragma unroll
        for (int q = 0; q < kWords; q += 8)
            asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                         : "=r"(w[q]), "=r"(w[q + 1]), "=r"(w[q + 2]), "=r"(w[q + 3]), "=r"(w[q + 4]), "=r"(w[q + 5]),
                           "=r"(w[q + 6]), "=r"(w[q + 7])
                         : "l"(p + q * PW));
    }
    // 8-byte aligned, `left` values exist (zeros after them): the whole pieces of 8 bytes
    // first, for all steps, with no branch between them, then a last broken one
    static constexpr int kPiece = 8 / (int)sizeof(T);
    __device__ __forceinline__ void load_pieces(const T* p, int left) {
#pragma unroll
        for (int q = 0; q < kWords / 2; ++q) {
            const uint2 u = (q + 1) * kPiece <= left ? reinterpret_cast<const uint2*>(p)[q] : make_uint2(0u, 0u);
            w[2 * q] = u.x;
            w[2 * q + 1] = u.y;
        }
    }
    __device__ __forceinline__ void load_rest(const T* p, int left) {
        if (left <= 0 || left >= N || left % kPiece == 0) return;
#pragma unroll
        for (int t = 0; t < N; ++t)
            if (t >= left / kPiece * kPiece && t < left) w[t / PW] = with_part<T>(w[t / PW], t % PW, to_f32(p[t]));
    }
    // any alignment, one by one
    __device__ __forceinline__ void load_single(const T* p, int left) {
#pragma unroll
        for (int q = 0; q < kWords; ++q) {
            if (PW == 1) {
                w[q] = q < left ? reinterpret_cast<const uint32_t*>(p)[q] : 0u;
            } else {
                const uint16_t lo = 2 * q < left ? reinterpret_cast<const uint16_t*>(p)[2 * q] : (uint16_t)0;
                const uint16_t hi = 2 * q + 1 < left ? reinterpret_cast<const uint16_t*>(p)[2 * q + 1] : (uint16_t)0;
                w[q] = (uint32_t)lo | (uint32_t)hi << 16;
            }
        }
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int q = 0; q < kWords; ++q) w[q] = 0u;
    }
    // the bits of the largest magnitude as fp32 (infinity where there is one; NaN gives way)
    __device__ __forceinline__ uint32_t largest() const {
        uint32_t a = w[0] & kAbs;
#pragma unroll
        for (int q = 1; q < kWords; ++q) a = max_parts<T>(a, w[q] & kAbs);
        if (PW == 1) return a;
        return __float_as_uint(fmaxf(part_of<T>(a, 0), part_of<T>(a, 1)));
    }
    __device__ __forceinline__ void drop_infinities() {
#pragma unroll
        for (int t = 0; t < N; ++t)
            w[t / PW] = with_part<T>(w[t / PW], t % PW, finite_or_nan(part_of<T>(w[t / PW], t % PW)));
    }
    // the codes of values 4 q .. 4 q + 3
    __device__ __forceinline__ uint32_t encode(int q, float inverse) const {
        float v[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) v[t] = part_of<T>(w[(4 * q + t) / PW], (4 * q + t) % PW);
        return encode4(v, inverse);
    }
};

// Writes rows (values of a row contiguous, rows `ldx` apart): a block's values are
// read once, stay in registers as they came, and leave as codes. FAST: rows are
// 16-byte aligned and d is a multiple of 8; lanes past the data then load a place
// inside it and drop it, so that no branch parts the loads.
template <class T, bool SLOTS, bool FAST>
__global__ void __launch_bounds__(256)
    k_block8_write(const T* __restrict__ X, int n, int d, int64_t ldx, int width, const int64_t* __restrict__ slots,
                   int first, const int* __restrict__ claims, uint8_t* __restrict__ codes,
                   uint8_t* __restrict__ scales, int64_t rows, int pitch, FastDiv nb, int* status) {
    pdl_wait();
    pdl_release();
    const int lane = threadIdx.x & 31, half = lane >> 4, col8 = (lane & 15) * 8;
    const uint32_t total = (uint32_t)n * nb.div;
    const uint32_t stride = gridDim.x * (blockDim.x >> 5) * kPairsPerWarp;
    const int groups = (int)(nb.div + 3) / 4;
    for (uint32_t f0 = (blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5)) * kPairsPerWarp; f0 < total; f0 += stride) {
        const Pairs at(f0 + half, nb);
        Values<T, 8> v[kSteps];
        int to[kSteps];
        if (FAST) {
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
                v[s].load16(X + (int64_t)min(at.row[s], n - 1) * ldx + min(at.b[s] * kBlock + col8, d - 8));
        } else {
            const T* src[kSteps];
            int left[kSteps];
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                const int col = at.b[s] * kBlock + col8;
                src[s] = X + (int64_t)at.row[s] * ldx + col;
                left[s] = at.row[s] < n ? d - col : 0;
            }
            if (width > 1) {
#pragma unroll
                for (int s = 0; s < kSteps; ++s) v[s].load_pieces(src[s], left[s]);
#pragma unroll
                for (int s = 0; s < kSteps; ++s) v[s].load_rest(src[s], left[s]);
            } else {
#pragma unroll
                for (int s = 0; s < kSteps; ++s) v[s].load_single(src[s], left[s]);
            }
        }
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            to[s] = -1;
            if (at.row[s] < n) to[s] = SLOTS ? (int)slot_of(slots, 0, at.row[s], rows, status) : first + at.row[s];
        }
        int mine = 0, my_to = -1, my_b = 0;  // lane 16 half + s keeps the exponent of step s
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const int col = at.b[s] * kBlock + col8;
            if (SLOTS && !last_of_slot(slots, claims, at.row[s], n, to[s], lane & 15, 16)) to[s] = -1;
            if (FAST && col >= d) v[s].clear();
            uint32_t a = v[s].largest();
            uint32_t lo = __reduce_max_sync(0xFFFFFFFFu, half ? 0u : a), hi = __reduce_max_sync(0xFFFFFFFFu, half ? a : 0u);
            if (max(lo, hi) >= 0x7F800000u) {  // an infinity (or NaN alone): held as NaN, the block scaled by the others
                v[s].drop_infinities();
                a = v[s].largest();
                if (a >= 0x7F800000u) a = 0u;  // NaN alone
                lo = __reduce_max_sync(0xFFFFFFFFu, half ? 0u : a);
                hi = __reduce_max_sync(0xFFFFFFFFu, half ? a : 0u);
            }
            const int e = block_exponent(half ? hi : lo);
            const float inverse = __uint_as_float((uint32_t)(127 - e) << 23);
            if (to[s] >= 0 && col < pitch)
                *reinterpret_cast<uint2*>(codes + (int64_t)to[s] * pitch + col) =
                    make_uint2(v[s].encode(0, inverse), v[s].encode(1, inverse));
            if ((lane & 15) == s) {
                mine = e + 127;
                my_to = to[s];
                my_b = at.b[s];
            }
        }
        if (my_to >= 0) scales[scale_at(my_to, my_b, groups)] = (uint8_t)mine;
    }
}

// The same where d is a multiple of 16 and the rows of X are 32-byte aligned: 16 values
// per lane, 8 lanes per pair, two steps of four pairs in flight. With 8 values per lane
// the work to find them kept 16-bit inputs from the memory's rate (65,536 x 768 bf16
// 29 us).
template <class T, bool SLOTS>
__global__ void __launch_bounds__(256)
    k_block8_write_wide(const T* __restrict__ X, int n, int d, int64_t ldx, const int64_t* __restrict__ slots, int first,
                        const int* __restrict__ claims, uint8_t* __restrict__ codes, uint8_t* __restrict__ scales,
                        int64_t rows, FastDiv nb, int* status) {
    pdl_wait();
    pdl_release();
    constexpr int kWideSteps = 2;
    static_assert(4 * kWideSteps == kPairsPerWarp, "the launch shape of k_block8_write");
    const int lane = threadIdx.x & 31, part = lane >> 3, col16 = (lane & 7) * 16;
    const uint32_t total = (uint32_t)n * nb.div;
    const uint32_t stride = gridDim.x * (blockDim.x >> 5) * kPairsPerWarp;
    const int groups = (int)(nb.div + 3) / 4;
    for (uint32_t f0 = (blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5)) * kPairsPerWarp; f0 < total; f0 += stride) {
        Values<T, 16> v[kWideSteps];
        int row[kWideSteps], b[kWideSteps], to[kWideSteps];
#pragma unroll
        for (int s = 0; s < kWideSteps; ++s) {  // (lanes past the data load a place inside it and drop it)
            const uint32_t f = f0 + 4 * s + part;
            row[s] = (int)nb.quotient(f);
            b[s] = (int)(f - (uint32_t)row[s] * nb.div);
            v[s].load32(X + (int64_t)min(row[s], n - 1) * ldx + min(b[s] * kBlock + col16, d - 16));
        }
#pragma unroll
        for (int s = 0; s < kWideSteps; ++s) {
            to[s] = -1;
            if (row[s] < n) to[s] = SLOTS ? (int)slot_of(slots, 0, row[s], rows, status) : first + row[s];
        }
        int mine = 0, my_to = -1, my_b = 0;  // lane 8 part + s keeps the exponent of step s
#pragma unroll
        for (int s = 0; s < kWideSteps; ++s) {
            const int col = b[s] * kBlock + col16;
            if (SLOTS && !last_of_slot(slots, claims, row[s], n, to[s], lane & 7, 8)) to[s] = -1;
            if (col >= d) v[s].clear();
            uint32_t a = v[s].largest();
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) a = max(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
            if (__any_sync(0xFFFFFFFFu, a >= 0x7F800000u)) {  // (as in k_block8_write)
                v[s].drop_infinities();
                a = v[s].largest();
                if (a >= 0x7F800000u) a = 0u;  // NaN alone
#pragma unroll
                for (int o = 4; o > 0; o >>= 1) a = max(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
            }
            const int e = block_exponent(a);
            const float inverse = __uint_as_float((uint32_t)(127 - e) << 23);
            if (to[s] >= 0 && col < d)
                *reinterpret_cast<uint4*>(codes + (int64_t)to[s] * d + col) =
                    make_uint4(v[s].encode(0, inverse), v[s].encode(1, inverse), v[s].encode(2, inverse),
                               v[s].encode(3, inverse));
            if ((lane & 7) == s) {
                mine = e + 127;
                my_to = to[s];
                my_b = b[s];
            }
        }
        if (my_to >= 0) scales[scale_at(my_to, my_b, groups)] = (uint8_t)mine;
    }
}

// Writes rows given as columns: value j of row i is X[j * ldx + i], so consecutive
// rows are contiguous in memory. A block of 256 threads takes a tile of one block of
// 128 values x kRows rows, 128 bytes of X for each value: a thread loads 16 bytes (V
// rows) of 4 consecutive values, so that its codes of a row are one word. The rows'
// maxima (of 16-bit types two to a word) meet by shuffles and in shared memory; the
// words are turned in shared memory (16-byte pieces of a row XORed with the row's group
// of V, which keeps both sides off each other's banks) and leave as 128 bytes per row.
// The values stay in their type and a row's exponent is found by one thread, so that five
// blocks share an SM on 48 registers (fp32: six, on 40): 1,000 rows of 30,001 fp16 values
// take 19 us (with the values kept as floats, 100 registers, and every thread finding the
// exponents 46). Columns whose distance is no multiple of 16 bytes are loaded value by
// value: 4,095 rows of 16,384 bf16 79 us, 4,096 of them 40 (fp32 61 and 53).
template <class T>
struct ColTile {
    static constexpr int V = 16 / (int)sizeof(T);
    static constexpr int kRows = 8 * V;
    static constexpr int kPerWord = 4 / (int)sizeof(T);
    static constexpr uint32_t kAbs = sizeof(T) == 4 ? 0x7FFFFFFFu : 0x7FFF7FFFu;
    // (4,096 rows of 16,384 values: fp32 with 6 blocks on an SM 51.6 us, with 5 54.3; bf16
    // with 5 38.0, with 6, on 40 registers, 40.3)
    static constexpr int kBlocksPerSm = sizeof(T) == 4 ? 6 : 5;
};

template <class T>
__global__ void __launch_bounds__(256, ColTile<T>::kBlocksPerSm)
    k_block8_write_cols(const T* __restrict__ X, int n, int d, int64_t ldx, int width,
                        const int64_t* __restrict__ slots, int64_t first, const int* __restrict__ claims,
                        uint8_t* __restrict__ codes, uint8_t* __restrict__ scales, int64_t rows, int pitch,
                        FastDiv row_tiles, int* status) {
    using C = ColTile<T>;
    constexpr int V = C::V, kRows = C::kRows, PW = C::kPerWord;
    __shared__ __align__(16) uint32_t amax[8][kRows / PW];
    __shared__ __align__(16) uint8_t turned[kRows * kBlock];
    __shared__ __align__(16) float inverse[kRows];  // 2^-e of the tile's rows
    __shared__ int dest[kRows];
    pdl_wait();
    pdl_release();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int k = threadIdx.x & 7, jq = threadIdx.x >> 3;  // which V rows, which 4 values
    const int nb = (d + kBlock - 1) / kBlock, groups = (nb + 3) / 4;
    const uint32_t tiles = row_tiles.div * (uint32_t)nb;
    for (uint32_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int b = (int)row_tiles.quotient(t), base = (int)(t - (uint32_t)b * row_tiles.div) * kRows;
        const int i0 = base + V * k, j0 = b * kBlock + 4 * jq;
        const T* src = X + (int64_t)j0 * ldx + i0;
        uint32_t x[4][4];
        if (width == V && i0 + V <= n && j0 + 4 <= d) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint4 u = *reinterpret_cast<const uint4*>(src + q * ldx);
                x[q][0] = u.x; x[q][1] = u.y; x[q][2] = u.z; x[q][3] = u.w;
            }
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int r = 0; r < V; ++r) {
                    const float f = j0 + q < d && i0 + r < n ? to_f32(src[q * ldx + r]) : 0.0f;
                    x[q][r / PW] = with_part<T>(r % PW ? x[q][r / PW] : 0u, r % PW, f);
                }
        }
        // where the tile's rows go
        if (slots)
            for (int r = w; r < kRows; r += 8) {
                const int i = base + r;
                int64_t to = i < n ? slot_of(slots, first, i, rows, status) : -1;
                if (!last_of_slot(slots, claims, i, n, to, lane, 32)) to = -1;
                if (lane == 0) dest[r] = (int)to;
            }
        uint32_t a[4], top = 0u;
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            a[h] = 0u;
#pragma unroll
            for (int q = 0; q < 4; ++q) a[h] = max_parts<T>(a[h], x[q][h] & C::kAbs);
            top = max_parts<T>(top, a[h]);
        }
        if (isinf(part_of<T>(top, 0)) || isinf(part_of<T>(top, PW - 1))) {
            // an infinity: held as NaN, the block scaled by the others
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                a[h] = 0u;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
#pragma unroll
                    for (int s = 0; s < PW; ++s)
                        x[q][h] = with_part<T>(x[q][h], s, finite_or_nan(part_of<T>(x[q][h], s)));
                    a[h] = max_parts<T>(a[h], x[q][h] & C::kAbs);
                }
            }
        }
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            a[h] = max_parts<T>(a[h], __shfl_xor_sync(0xFFFFFFFFu, a[h], 8));
            a[h] = max_parts<T>(a[h], __shfl_xor_sync(0xFFFFFFFFu, a[h], 16));
        }
        if (lane < 8) *reinterpret_cast<uint4*>(&amax[w][4 * k]) = make_uint4(a[0], a[1], a[2], a[3]);
        __syncthreads();
        if (threadIdx.x < kRows / PW) {  // one thread per word of maxima: the rows' exponents
            const int i = PW * threadIdx.x;
            uint32_t m = amax[0][threadIdx.x];
#pragma unroll
            for (int q = 1; q < 8; ++q) m = max_parts<T>(m, amax[q][threadIdx.x]);
#pragma unroll
            for (int r = 0; r < PW; ++r) {
                const int e = block_exponent(__float_as_uint(part_of<T>(m, r)));
                inverse[i + r] = __uint_as_float((uint32_t)(127 - e) << 23);
                const int to = slots ? dest[i + r] : base + i + r < n ? (int)first + base + i + r : -1;
                if (to >= 0) scales[scale_at(to, b, groups)] = (uint8_t)(e + 127);
            }
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < V; ++r) {
            const float v[4] = {part_of<T>(x[0][r / PW], r % PW), part_of<T>(x[1][r / PW], r % PW),
                                part_of<T>(x[2][r / PW], r % PW), part_of<T>(x[3][r / PW], r % PW)};
            *reinterpret_cast<uint32_t*>(turned + (V * k + r) * kBlock + 4 * (jq ^ (4 * k))) =
                encode4(v, inverse[V * k + r]);
        }
        __syncthreads();
        // 8 threads per row, 16 codes each
#pragma unroll
        for (int q = 0; q < kRows / 32; ++q) {
            const int r = (threadIdx.x >> 3) + 32 * q, c = threadIdx.x & 7;
            const int to = slots ? dest[r] : base + r < n ? (int)first + base + r : -1;
            if (to >= 0 && b * kBlock + 16 * c < pitch)
                *reinterpret_cast<uint4*>(codes + (int64_t)to * pitch + b * kBlock + 16 * c) =
                    *reinterpret_cast<const uint4*>(turned + r * kBlock + 16 * (c ^ (r / V)));
        }
        __syncthreads();
    }
}

// Reads rows back, pairs as in k_block8_write. Exact in fp32 and bf16; fp16 rounds to
// nearest even (and overflows to infinity). Padding rows (slot -1) and rows outside
// the matrix read as zeros. `columns` values are written for each row, zeros past d.
// What bounds it is issue: 8 values are 27 instructions to load, decode, scale and
// store, and finding them must not cost as much again (32-bit row numbers, the next
// pair by steps, no branch between the loads).
template <class T, bool SLOTS>
__global__ void __launch_bounds__(256, 5)
    k_block8_read(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t rows, int pitch,
                  int d, const int64_t* __restrict__ slots, int first, int n, T* __restrict__ out, int64_t ldo,
                  int columns, int width, FastDiv nb, int* status) {
    pdl_wait();
    pdl_release();
    const int lane = threadIdx.x & 31, half = lane >> 4, col8 = (lane & 15) * 8;
    const uint32_t total = (uint32_t)n * nb.div;
    const uint32_t stride = gridDim.x * (blockDim.x >> 5) * kPairsPerWarp;
    const int groups = (int)(nb.div + 3) / 4;
    for (uint32_t f0 = (blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5)) * kPairsPerWarp; f0 < total; f0 += stride) {
        const Pairs at(f0 + half, nb);
        uint2 c[kSteps];
        uint8_t byte[kSteps];
        int from[kSteps];
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            from[s] = -1;
            if (at.row[s] < n) from[s] = SLOTS ? (int)slot_of(slots, 0, at.row[s], rows, status) : first + at.row[s];
        }
        // (a row that is left out loads row 0 and drops it, so that no branch parts the loads)
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const int r = max(from[s], 0);
            c[s] = *reinterpret_cast<const uint2*>(codes + (int64_t)r * pitch + min(at.b[s] * kBlock + col8, pitch - 8));
            byte[s] = scales[scale_at(r, at.b[s], groups)];
        }
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            if (at.row[s] >= n) break;
            const int col = at.b[s] * kBlock + col8;
            if (from[s] < 0) c[s] = make_uint2(0u, 0u);
            const float scale = scale_of(byte[s]);
            float v[8];
            decode4(c[s].x, v);
            decode4(c[s].y, v + 4);
#pragma unroll
            for (int t = 0; t < 8; ++t) v[t] *= scale;
            T* dst = out + (int64_t)at.row[s] * ldo + col;
            if (col + 8 > d) {
#pragma unroll
                for (int t = 0; t < 8; ++t) v[t] = col + t < d ? v[t] : 0.0f;
            }
            store8(dst, columns - col, width, v);
        }
    }
}

// The same where d is a multiple of 16 and the output's rows are 32-byte aligned: 16
// values per lane, 8 lanes per pair, two steps of four pairs in flight, and 32-byte
// stores. A lane's work to find its values is shared by twice as many. 32 registers, so
// that an SM is full of warps (65,536 rows of 768 gathered to bf16: 27.2 us, with 40 of
// its 64 warps 30.0).
__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

template <class T, bool SLOTS>
__global__ void __launch_bounds__(256, 8)
    k_block8_read_wide(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t rows, int d,
                       const int64_t* __restrict__ slots, int first, int n, T* __restrict__ out, int64_t ldo, FastDiv nb,
                       int* status) {
    pdl_wait();
    pdl_release();
    constexpr int kWideSteps = 2;
    static_assert(4 * kWideSteps == kPairsPerWarp, "the launch shape of k_block8_read");
    const int lane = threadIdx.x & 31, part = lane >> 3, col16 = (lane & 7) * 16;
    const uint32_t total = (uint32_t)n * nb.div;
    const uint32_t stride = gridDim.x * (blockDim.x >> 5) * kPairsPerWarp;
    const int groups = (int)(nb.div + 3) / 4;
    for (uint32_t f0 = (blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5)) * kPairsPerWarp; f0 < total; f0 += stride) {
        uint4 c[kWideSteps];
        uint8_t byte[kWideSteps];
        int row[kWideSteps], b[kWideSteps], from[kWideSteps];
#pragma unroll
        for (int s = 0; s < kWideSteps; ++s) {
            const uint32_t f = f0 + 4 * s + part;
            row[s] = (int)nb.quotient(f);
            b[s] = (int)(f - (uint32_t)row[s] * nb.div);
            from[s] = -1;
            if (f < total) from[s] = SLOTS ? (int)slot_of(slots, 0, row[s], rows, status) : first + row[s];
        }
#pragma unroll
        for (int s = 0; s < kWideSteps; ++s) {  // (as in k_block8_read: no branch parts the loads; d is the pitch)
            const int r = max(from[s], 0);
            c[s] = *reinterpret_cast<const uint4*>(codes + (int64_t)r * d + min(b[s] * kBlock + col16, d - 16));
            byte[s] = scales[scale_at(r, b[s], groups)];
        }
#pragma unroll
        for (int s = 0; s < kWideSteps; ++s) {
            const int col = b[s] * kBlock + col16;
            if (f0 + 4 * s + part >= total || col >= d) continue;
            if (from[s] < 0) c[s] = make_uint4(0u, 0u, 0u, 0u);
            const float scale = scale_of(byte[s]);
            const uint32_t cw[4] = {c[s].x, c[s].y, c[s].z, c[s].w};
            uint32_t w[8];
            T* dst = out + (int64_t)row[s] * ldo + col;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float v[4];
                decode4(cw[q], v);
                if (sizeof(T) == 4) {
#pragma unroll
                    for (int t = 0; t < 4; ++t) w[4 * (q & 1) + t] = __float_as_uint(v[t] * scale);
                    if (q & 1) store32(dst + 8 * (q >> 1), w);
                } else {
#pragma unroll
                    for (int t = 0; t < 4; t += 2) {
                        const T lo = from_f32<T>(v[t] * scale), hi = from_f32<T>(v[t + 1] * scale);
                        uint16_t l, h;
                        memcpy(&l, &lo, 2);
                        memcpy(&h, &hi, 2);
                        w[2 * q + t / 2] = (uint32_t)l | ((uint32_t)h << 16);
                    }
                    if (q == 3) store32(dst, w);
                }
            }
        }
    }
}

// The same to rows that no vector store can reach: a warp takes whole blocks, four
// consecutive (row, block) pairs at a time, and a lane the values lane, lane + 32, lane
// + 64 and lane + 96 of each, so that every store of a warp is one run of neighbours.
// (With 8 consecutive values per lane, stored one by one, 30,000 rows of 1,581 fp16
// values took 132 us in order and 129 by slots, and here 54 and 78; of 1,579 fp32 values
// 153 and 144, and here 57 and 73.)
struct BlockPairs {
    int row[kSteps], b[kSteps];
    __device__ __forceinline__ BlockPairs(uint32_t f, const FastDiv& nb) {
        row[0] = (int)nb.quotient(f);
        b[0] = (int)(f - (uint32_t)row[0] * nb.div);
#pragma unroll
        for (int s = 1; s < kSteps; ++s) {
            const bool next = b[s - 1] + 1 == (int)nb.div;
            b[s] = next ? 0 : b[s - 1] + 1;
            row[s] = row[s - 1] + (next ? 1 : 0);
        }
    }
};

template <class T, bool SLOTS>
__global__ void __launch_bounds__(256)
    k_block8_read_any(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t rows, int pitch,
                      int d, const int64_t* __restrict__ slots, int first, int n, T* __restrict__ out, int64_t ldo,
                      int columns, FastDiv nb, int* status) {
    pdl_wait();
    pdl_release();
    const int lane = threadIdx.x & 31;
    const uint32_t total = (uint32_t)n * nb.div;
    const uint32_t stride = gridDim.x * (blockDim.x >> 5) * kSteps;
    const int groups = (int)(nb.div + 3) / 4;
    for (uint32_t f0 = (blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5)) * kSteps; f0 < total; f0 += stride) {
        const BlockPairs at(f0, nb);
        uint8_t c[kSteps][4], byte[kSteps];
        int from[kSteps];
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            from[s] = -1;
            if (at.row[s] < n) from[s] = SLOTS ? (int)slot_of(slots, 0, at.row[s], rows, status) : first + at.row[s];
        }
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const int r = max(from[s], 0), col = at.b[s] * kBlock + lane, left = from[s] < 0 ? 0 : pitch - col;
            const uint8_t* src = codes + (int64_t)r * pitch + col;
#pragma unroll
            for (int t = 0; t < 4; ++t) c[s][t] = 32 * t < left ? src[32 * t] : (uint8_t)0;
            byte[s] = scales[scale_at(r, at.b[s], groups)];
        }
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            if (at.row[s] >= n) break;
            const int col = at.b[s] * kBlock + lane;
            const float scale = scale_of(byte[s]);
            float v[4];
            decode4((uint32_t)c[s][0] | (uint32_t)c[s][1] << 8 | (uint32_t)c[s][2] << 16 | (uint32_t)c[s][3] << 24, v);
            T* dst = out + (int64_t)at.row[s] * ldo + col;
            const int left = columns - col, held = d - col;
#pragma unroll
            for (int t = 0; t < 4; ++t)
                if (32 * t < left) dst[32 * t] = from_f32<T>(32 * t < held ? v[t] * scale : 0.0f);
        }
    }
}

// ---------------------------------------------------------------- product
//
// out = A B^T of two block8 matrices on the tensor cores' block-scaled FP8 path
// (tcgen05.mma kind::mxf8f6f4, fp32 accumulators): the scales enter the MMA as E8M0
// factors, so a product of held values is exact and only the accumulation rounds.
// The hardware takes one factor per 32 values of a row; the four K = 32 steps of a
// block name the same byte (the scale-factor id of the instruction descriptor picks
// byte block % 4 of the row's word), so one stored byte serves 128 values.
//
// The MMA's own accumulation cuts off below fp32's last place instead of rounding, an
// error that grows with the number of steps (5.7e-7 of the result at d = 4096). So a
// contraction is cut into spans of kSpan blocks: each starts a fresh accumulator, and
// the epilogue adds the spans in order, rounding to nearest, in registers. Two
// accumulators let it read one while the next span runs.
//
// Roles of a CTA's warps:
//   warps 0, 2 load A and B: 128-byte-wide tiles of codes (TMA, 128-byte swizzle) and
//              the exponents of their rows into a ring of stages (one warp for both took
//              a block's loads as long to issue as its MMAs run)
//   warp 1     one thread issues the MMAs and, at every fourth block of a row, copies the
//              exponents of four blocks to tensor memory. They go round as many sets of
//              columns there as the ring has blocks: a set's last user is at least that
//              many blocks back, and the wait for this block's stage was a wait for it
//   from 3 on  epilogue: groups of four warps, one per TMEM lane quadrant, each with its
//              columns of a tile

constexpr int kMmThreads = 352;
constexpr int kSpan = 8;                      // blocks of 128 values per accumulator
constexpr int kTurnBytes = 8 * 32 * 128;      // epilogue warps' turning buffers
constexpr int kCodeTile = 128 * 128;          // codes of 128 rows x one block

template <bool CLUSTER>
__device__ __forceinline__ bool try_bar(uint32_t bar, uint32_t parity) {
    if (!CLUSTER) return tc::mbar_try_wait(bar, parity);
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// Waits for a phase of `bar` (CLUSTER: the other CTA of the pair may arrive on it);
// after `limit` clock cycles it raises EM_E_TIMEOUT and the CTA's abort flag and gives
// up. (An error that an earlier call left in the matrix's status word, an out-of-range
// slot say, does not stop a product: only this CTA's own waits do.)
template <bool CLUSTER = false>
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, long long limit, int* status,
                                         volatile int* abort_flag) {
    if (try_bar<CLUSTER>(bar, parity)) return true;
    const long long t0 = clock64();
    for (uint32_t it = 1;; ++it) {
        if (try_bar<CLUSTER>(bar, parity)) return true;
        if ((it & 63u) == 0) {
            if (*abort_flag) return false;
            if (clock64() - t0 > limit) {
                raise_error(status, EM_E_TIMEOUT);
                *abort_flag = 1;
                return false;
            }
        }
    }
}

// wait_bar by a whole warp, with one vote where the phase is complete already.
template <bool CLUSTER = false>
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, long long limit, int* status,
                                          volatile int* abort_flag) {
    if (__all_sync(0xFFFFFFFFu, try_bar<CLUSTER>(bar, parity))) return true;
    return __all_sync(0xFFFFFFFFu, wait_bar<CLUSTER>(bar, parity, limit, status, abort_flag));
}

// Self-test of the failure path (em_selftest 3): two warps wait on a barrier that
// nothing arrives on; one reaches its limit, the other sees the abort flag.
__global__ void k_block8_selftest(long long limit, int* status) {
    __shared__ __align__(8) uint64_t bar;
    __shared__ int abort_flag;
    if (threadIdx.x == 0) {
        abort_flag = 0;
        tc::mbar_init(tc::smem_u32(&bar), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    // the second warp's own limit is far beyond the first's
    wait_bar<true>(tc::smem_u32(&bar), 0u, threadIdx.x < 32 ? limit : 64 * limit, status, &abort_flag);
}

// One lane of a converged warp. The issuing warps walk their loops with all lanes and
// let one issue: the loop's values stay warp-uniform, and the MMA's operands with them
// (under a branch on the lane the issue itself took longer than the MMAs).
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xFFFFFFFF;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(r));
    return r != 0;
}

// Instruction descriptor of tcgen05.mma kind::mxf8f6f4: the scale-factor ids in bits
// 4-5 (B) and 29-30 (A), E4M3 operands (format 0 in bits 7-9 and 10-12), K-major (bits
// 15, 16 = 0), N >> 3 in bits 17-22, E8M0 scales (bit 23), M >> 7 in bits 27-28.
__device__ __forceinline__ uint32_t mm_idesc(int m, int n, uint32_t sf_id) {
    return (sf_id << 4) | ((uint32_t)(n >> 3) << 17) | (1u << 23) | ((uint32_t)(m >> 7) << 27) | (sf_id << 29);
}

template <int CG>
__device__ __forceinline__ void umma_block8(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                            uint32_t sfb, uint32_t accumulate) {
    if (CG == 1)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(d_tmem),
            "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(d_tmem),
            "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
}

// 512 bytes of exponents to four tensor-memory columns, repeated in each lane
// quadrant (CG = 2: in each CTA of the pair, from its own shared memory). The
// descriptor: no swizzle, 8-row groups of 16-byte rows 128 bytes apart.
template <int CG>
__device__ __forceinline__ void copy_exponents(uint32_t tmem, uint32_t smem) {
    if (CG == 1)
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem),
                     "l"(tc::smem_desc(smem, 0ull, 128u))
                     : "memory");
    else
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem),
                     "l"(tc::smem_desc(smem, 0ull, 128u))
                     : "memory");
}

struct MmArgs {
    void* out;
    int64_t ldo;
    int64_t m_rows, n_rows;  // rows of the M and N operands that the product takes
    int nkb;                 // blocks along the rows
    int m_tiles, n_tiles;
    int split;               // CTAs (a cluster) that share a tile, one span each; 1: none do
    int bf16;                // 16-bit results: bf16 rather than fp16
    int vec_ok;              // 16-byte aligned output rows
    long long wait_limit;
    int* status;
};

// At least about 2 s, whatever limit the waits had.
__device__ __forceinline__ long long drain_limit(const MmArgs& p) { return max(p.wait_limit, 4000000000ll); }

// The end of a CTA that gave up: its shared and tensor memory go to the next one, so that
// every load of the ring must have landed, whichever role gave up and wherever the loaders
// stood. `begun`: fills of the loader that is ahead. A fill that another loader did not
// begin never completes; `limit` cycles, for all fills together, end the wait for it, a
// million times what a load takes.
template <int S>
__device__ __forceinline__ void drain_ring(const uint64_t* full, uint32_t begun, long long limit) {
    const long long t0 = clock64();
    for (uint32_t i = ring_first(begun, S); i != begun; ++i)
        tc::mbar_drain(tc::smem_u32(&full[ring_stage(i, S)]), ring_parity(i, S), max(limit - (clock64() - t0), 0ll));
}

__device__ __forceinline__ uint32_t pack_out(uint32_t lo, uint32_t hi, int bf16) {
    uint32_t r;
    if (bf16) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(__uint_as_float(lo), __uint_as_float(hi));
        memcpy(&r, &p, 4);
    } else {
        const __half2 p = __floats2half2_rn(__uint_as_float(lo), __uint_as_float(hi));
        memcpy(&r, &p, 4);
    }
    return r;
}

// Running sums of a lane's row start at -0, to which the first span adds exactly.
// (Setting them from the first span instead made the compiler keep two copies.)
template <int NS>
__device__ __forceinline__ void clear_sums(uint32_t (&sum)[NS][32]) {
#pragma unroll
    for (int i = 0; i < NS; ++i)
#pragma unroll
        for (int e = 0; e < 32; ++e) sum[i][e] = 0x80000000u;
}

// Adds 32 accumulator columns of this lane's row to its running sums.
__device__ __forceinline__ void add_columns(uint32_t taddr, uint32_t (&sum)[32]) {
#pragma unroll
    for (int h = 0; h < 32; h += 16) {
        uint32_t v[16];
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
            "%15}, [%16];\n\ttcgen05.wait::ld.sync.aligned;"
            : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
              "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
            : "r"(taddr + h)
            : "memory");
#pragma unroll
        for (int i = 0; i < 16; ++i)
            sum[h + i] = __float_as_uint(__uint_as_float(sum[h + i]) + __uint_as_float(v[i]));
    }
}

// One warp's 32 rows x Q 16-byte pieces of results (lane = row, 4 Q words w) to rows
// row0.. and columns col0.. of `out`: turned in the warp's 4 KB of shared memory (a
// piece's place in its row XORed with the row, so that neither side meets a bank
// twice), then stored as whole row pieces, Q lanes to a row.
template <int OB, int Q>
__device__ __forceinline__ void store_piece(const uint32_t (&w)[32], uint8_t* buf, int lane, int64_t row0, int64_t col0,
                                            const MmArgs& p) {
    if (col0 >= p.n_rows) return;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < Q; ++i)
        *reinterpret_cast<uint4*>(buf + lane * 128 + ((i ^ (lane & 7)) << 4)) =
            make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    __syncwarp();
    constexpr int kPer = 16 / OB;  // columns of a piece
    if (p.vec_ok && col0 + Q * kPer <= p.n_rows) {
        constexpr int kRows = 32 / Q;  // rows per step
        const int piece = lane % Q, r0 = lane / Q;
        uint8_t* dst = reinterpret_cast<uint8_t*>(p.out) + ((row0 + r0) * p.ldo + col0 + piece * kPer) * OB;
#pragma unroll
        for (int i = 0; i < Q; ++i) {
            const int r = kRows * i + r0;
            const uint4 x = *reinterpret_cast<const uint4*>(buf + r * 128 + ((piece ^ (r & 7)) << 4));
            if (row0 + r < p.m_rows) *reinterpret_cast<uint4*>(dst) = x;
            dst += kRows * p.ldo * OB;
        }
        return;
    }
    // rows that are not 16-byte aligned, or end inside: 32 neighbouring columns at a time
    const int rows = (int)min(p.m_rows - row0, (int64_t)32), cols = (int)min(p.n_rows - col0, (int64_t)(Q * kPer));
#pragma unroll 1
    for (int r = 0; r < rows; ++r) {
        uint8_t* dst = reinterpret_cast<uint8_t*>(p.out) + ((row0 + r) * p.ldo + col0) * OB;
#pragma unroll
        for (int c = lane; c < Q * kPer; c += 32) {
            const uint8_t* x = buf + r * 128 + (((c / kPer) ^ (r & 7)) << 4) + c % kPer * OB;
            if (c < cols) {
                if (OB == 4)
                    reinterpret_cast<uint32_t*>(dst)[c] = *reinterpret_cast<const uint32_t*>(x);
                else
                    reinterpret_cast<uint16_t*>(dst)[c] = *reinterpret_cast<const uint16_t*>(x);
            }
        }
    }
}

// A lane's NS x 32 results from column col0 on.
template <int OB, int NS>
__device__ __forceinline__ void store_rows(const uint32_t (&sum)[NS][32], uint8_t* buf, int lane, int64_t row0,
                                           int64_t col0, const MmArgs& p) {
    if (OB == 4) {
#pragma unroll
        for (int i = 0; i < NS; ++i) store_piece<OB, 8>(sum[i], buf, lane, row0, col0 + 32 * i, p);
    } else {
#pragma unroll
        for (int i = 0; i < NS; i += 2) {
            uint32_t w[32];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                w[e] = pack_out(sum[i][2 * e], sum[i][2 * e + 1], p.bf16);
                if (i + 1 < NS) w[16 + e] = pack_out(sum[i + 1 < NS ? i + 1 : i][2 * e], sum[i + 1 < NS ? i + 1 : i][2 * e + 1], p.bf16);
            }
            if (i + 1 < NS)
                store_piece<OB, 8>(w, buf, lane, row0, col0 + 32 * i, p);
            else
                store_piece<OB, 4>(w, buf, lane, row0, col0 + 32 * i, p);
        }
    }
}

// ---- one CTA per 128 x BN tile: few tiles, or few rows on one side
//
// SWAP: the M operand is the one whose rows are the output's columns (few output
// rows): a lane holds one output column and a warp stores 32 neighbours at once.
// With few rows on one side the product streams the long operand once, and what counts
// is bytes in flight: BN = 32 keeps the stages small and lets two groups of four
// epilogue warps take tiles in turn, four accumulators ahead (300,000 rows of 128 with
// 24 others: 15 us where they are the columns of the result; where they are its rows 28,
// and 66 in 256 x 192 tiles).
//
// The blocks of all of a CTA's tiles form one sequence, PER of them to a stage: a
// barrier round trip serves PER blocks whatever the rows' length.
//
// Long rows with few tiles: a cluster of `split` CTAs shares a tile, one span of the
// rows each. The spans' results meet in shared memory, and the cluster's first CTA adds
// them in order: the sums are those of a CTA that does all spans, bit for bit. A cluster
// has at most 8 CTAs; longer rows, and more tiles than SMs / spans, have a CTA to a tile
// (16 x 512: d = 8,192 7.9 us, 8,193 18.5, 16,384 33; 1,024 x 512 x 16,384 40).

template <int BN, bool SWAP>
struct MmCfg {
    static constexpr int kPer = SWAP || BN == 32 ? 2 : 1;
    static constexpr int kStages = BN == 32 ? (SWAP ? 5 : 4) : (SWAP ? 3 : 5);
    static constexpr int kBTile = BN * 128;
    static constexpr int kCodes = kCodeTile + kBTile;  // codes of one block
    static constexpr int kSf = 2 * kAtomBytes;
    static constexpr bool kTurns = BN == 32;           // the epilogue's halves take tiles in turn
    static constexpr int kAcc = kTurns ? 4 : 2;
    static constexpr int kSmem = 1024 + 256 + (SWAP ? 0 : kTurnBytes) + kStages * kPer * (kCodes + kSf);
    static constexpr int kSfCols = 8;
    static constexpr int kSfSlots = kStages * kPer;
    static constexpr int kSfBase = kAcc * BN;
    static_assert(kSmem <= 227 * 1024 && kSfBase + kSfSlots * kSfCols <= 512, "shared or tensor memory");
};

template <int BN, int OB, bool SWAP>
__global__ void __launch_bounds__(kMmThreads, 1)
    k_block8_matmul(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB, const MmArgs p) {
    using namespace tc;
    using C = MmCfg<BN, SWAP>;
    constexpr int S = C::kStages, PER = C::kPer, ACC = C::kAcc;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sA = smem;
    uint8_t* sB = sA + S * PER * kCodeTile;
    uint8_t* turn = sB + S * PER * C::kBTile;
    uint8_t* sSf = turn + (SWAP ? 0 : kTurnBytes);
    uint64_t* bars = reinterpret_cast<uint64_t*>(sSf + S * PER * C::kSf);
    uint64_t* full = bars;
    uint64_t* empty = bars + S;
    uint64_t* tfull = bars + 2 * S;
    uint64_t* tempty = tfull + ACC;
    uint64_t* drain = tempty + ACC;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    uint32_t* begun_by = tmem_slot + 2;  // stages that each loader began

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t tiles = (int64_t)p.m_tiles * p.n_tiles;
    const int groups = (p.nkb + 3) / 4;
    // this CTA's tiles and the blocks of their rows that it takes
    const bool shared_tile = p.split > 1;
    const int rank = shared_tile ? (int)(blockIdx.x % p.split) : 0;
    const int64_t first = shared_tile ? blockIdx.x / p.split : blockIdx.x, step = shared_tile ? tiles : gridDim.x;
    const int kb_lo = rank * kSpan, kb_hi = shared_tile ? min(p.nkb, kb_lo + kSpan) : p.nkb;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(smem_u32(&full[s]), 2 * PER);  // a load of A, one of B, for each block
            mbar_init(smem_u32(&empty[s]), 1);
        }
        for (int a = 0; a < ACC; ++a) {
            mbar_init(smem_u32(&tfull[a]), 1);
            mbar_init(smem_u32(&tempty[a]), C::kTurns ? 4 : 8);
        }
        mbar_init(smem_u32(drain), 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(512u)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    pdl_wait();
    pdl_release();

    if (warp == 0 || warp == 2) {
        const bool loads_a = warp == 0;
        int stage = 0, part = 0;  // the next block's stage, and its place there
        uint32_t phase = 0, begun = 0;
        bool ok = true;
        for (int64_t t = first; t < tiles && ok; t += step) {
            const int m = (int)(t / p.n_tiles), n = (int)(t - (int64_t)m * p.n_tiles);
            for (int kb = kb_lo; kb < kb_hi; ++kb) {
                if (part == 0) {
                    ok = wait_warp(smem_u32(&empty[stage]), phase ^ 1u, p.wait_limit, p.status, abort_flag);
                    if (!ok) break;
                    ++begun;
                }
                if (elect_one()) {
                    const uint32_t fb = smem_u32(&full[stage]);
                    const int at = stage * PER + part;
                    uint8_t* sf = sSf + at * C::kSf;
                    if (loads_a) {
                        mbar_expect_tx(fb, (uint32_t)(kCodeTile + ((kb & 3) == 0 ? kAtomBytes : 0)));
                        tma_load_2d(smem_u32(sA + at * kCodeTile), &tmA, kb * kBlock, m * 128, fb);
                        if ((kb & 3) == 0) tma_load_2d(smem_u32(sf), &tmSA, 0, m * groups + (kb >> 2), fb);
                    } else {
                        mbar_expect_tx(fb, (uint32_t)(C::kBTile + ((kb & 3) == 0 ? kAtomBytes : 0)));
                        tma_load_2d(smem_u32(sB + at * C::kBTile), &tmB, kb * kBlock, n * BN, fb);
                        if ((kb & 3) == 0) tma_load_2d(smem_u32(sf + kAtomBytes), &tmSB, 0, n * groups + (kb >> 2), fb);
                    }
                }
                __syncwarp();
                if (++part == PER) {
                    part = 0;
                    if (++stage == S) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
        }
        if (part > 0 && elect_one())  // the last stage's missing blocks
            for (; part < PER; ++part) mbar_arrive(smem_u32(&full[stage]));
        __syncwarp();
        if (lane == 0) begun_by[loads_a ? 0 : 1] = begun;
    } else if (warp == 1) {
        int stage = 0, part = 0, acc = 0, slot = C::kSfSlots - 1;
        uint32_t phase = 0, acc_phase = 0;
        bool ok = true;
        const uint64_t desc0 = smem_desc(0u, 2ull, 1024u);
        const uint32_t a_base = smem_u32(sA) >> 4, b_base = smem_u32(sB) >> 4;
        for (int64_t t = first; t < tiles && ok; t += step) {
            // four blocks share a group of exponents; unrolled, so that what the MMAs take
            // but a block's stage is fixed
            for (int kb0 = kb_lo; kb0 < kb_hi && ok; kb0 += 4) {
                if (kb0 % kSpan == 0)
                    ok = wait_warp(smem_u32(&tempty[acc]), acc_phase ^ 1u, p.wait_limit, p.status, abort_flag);
                if (++slot == C::kSfSlots) slot = 0;
                const uint32_t sf = tmem_base + (uint32_t)(C::kSfBase + slot * C::kSfCols);
                const uint32_t d_tmem = tmem_base + (uint32_t)(acc * BN);
                const int blocks = min(4, kb_hi - kb0);
                const bool last = kb0 % kSpan + 4 == kSpan || kb0 + blocks == kb_hi;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (i >= blocks) break;
                    if (part == 0)
                        ok = ok && wait_warp(smem_u32(&full[stage]), phase, p.wait_limit, p.status, abort_flag);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t at = (uint32_t)(stage * PER + part);
                    const uint32_t a_lo = a_base + at * (kCodeTile >> 4), b_lo = b_base + at * (C::kBTile >> 4);
                    if (elect_one()) {
                        if (i == 0) {
                            copy_exponents<1>(sf, smem_u32(sSf + at * C::kSf));
                            copy_exponents<1>(sf + 4, smem_u32(sSf + at * C::kSf + kAtomBytes));
                        }
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            umma_block8<1>(d_tmem, desc0 | (a_lo + 2 * kk), desc0 | (b_lo + 2 * kk),
                                           mm_idesc(128, BN, (uint32_t)i), sf, sf + 4,
                                           (i | kk) != 0 ? 1u : (uint32_t)(kb0 % kSpan));
                        if (part == PER - 1) umma_commit(smem_u32(&empty[stage]));
                        if (last && i == blocks - 1) umma_commit(smem_u32(&tfull[acc]));
                    }
                    __syncwarp();
                    if (++part == PER) {
                        part = 0;
                        if (++stage == S) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                }
                if (last && ++acc == ACC) {
                    acc = 0;
                    acc_phase ^= 1u;
                }
            }
        }
    }
    // ---------------- epilogue
    const int ew = warp - 3;
    const int q = warp & 3, half = ew >> 2;
    constexpr int kCols = C::kTurns ? BN : BN / 2;  // columns a warp takes
    constexpr int NS = kCols / 32;
    auto store = [&](const uint32_t (&sum)[NS][32], int64_t row0, int64_t col0) {
        if (SWAP) {
            const int64_t j = row0 + lane;  // output column
            const int rows = (int)min(p.n_rows - col0, (int64_t)kCols);
            uint8_t* dst = reinterpret_cast<uint8_t*>(p.out) + (col0 * p.ldo + j) * OB;
            if (j < p.m_rows) {
#pragma unroll
                for (int i = 0; i < NS; ++i)
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        if (32 * i + e < rows) {
                            if (OB == 4)
                                *reinterpret_cast<uint32_t*>(dst) = sum[i][e];
                            else
                                *reinterpret_cast<uint16_t*>(dst) = (uint16_t)pack_out(sum[i][e], 0u, p.bf16);
                        }
                        dst += p.ldo * OB;
                    }
            }
        } else {
            store_rows<OB, NS>(sum, turn + ew * 32 * 128, lane, row0, col0, p);
        }
    };
    // a shared tile's results of this CTA's span: [warp][column][lane], over the ring
    // (which is done with by the time the accumulator is complete)
    float* part = reinterpret_cast<float*>(sA) + ew * NS * 32 * 32 + lane;
    static_assert(8 * NS * 32 * 32 * 4 <= S * PER * kCodeTile, "the ring holds a tile's results");
    if (warp >= 3) {
        const uint32_t lane_base = (uint32_t)(32 * q) << 16;
        const int spans = shared_tile ? 1 : (p.nkb + kSpan - 1) / kSpan;
        int64_t span = C::kTurns ? (int64_t)half * spans : 0;  // spans of the CTA before this tile's
        bool ok = true;
        for (int64_t t = first + (C::kTurns ? half * step : 0); t < tiles && ok; t += (C::kTurns ? 2 : 1) * step) {
            const int m = (int)(t / p.n_tiles), n = (int)(t - (int64_t)m * p.n_tiles);
            uint32_t sum[NS][32];
            clear_sums(sum);
            for (int s = 0; s < spans; ++s) {
                const int acc = (int)(span % ACC);
                if (!wait_warp(smem_u32(&tfull[acc]), (uint32_t)(span / ACC) & 1u, p.wait_limit, p.status, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t tbase = tmem_base + lane_base + (uint32_t)(acc * BN + (C::kTurns ? 0 : half * kCols));
#pragma unroll
                for (int i = 0; i < NS; ++i) add_columns(tbase + 32 * i, sum[i]);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&tempty[acc]));
                ++span;
            }
            if (C::kTurns) span += spans;  // the other half's tile
            if (!ok) break;
            if (shared_tile) {
#pragma unroll
                for (int i = 0; i < NS; ++i)
#pragma unroll
                    for (int e = 0; e < 32; ++e) part[(32 * i + e) * 32] = __uint_as_float(sum[i][e]);
            } else {
                store(sum, (int64_t)m * 128 + 32 * q, (int64_t)n * BN + (C::kTurns ? 0 : half * kCols));
            }
        }
    }
    if (shared_tile) {
        __syncwarp();
        asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
        if (rank == 0 && warp >= 3 && (!C::kTurns || half == 0)) {
            uint32_t sum[NS][32];
            clear_sums(sum);
            for (int r = 0; r < p.split; ++r) {
                uint32_t from;
                asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(from) : "r"(smem_u32(part)), "r"(r));
#pragma unroll
                for (int i = 0; i < NS; ++i)
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        float v;
                        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(from + (32 * i + e) * 128) : "memory");
                        sum[i][e] = __float_as_uint(__uint_as_float(sum[i][e]) + v);
                    }
            }
            const int m = (int)(first / p.n_tiles), n = (int)(first - (int64_t)m * p.n_tiles);
            store(sum, (int64_t)m * 128 + 32 * q, (int64_t)n * BN + (C::kTurns ? 0 : half * kCols));
        }
        __syncwarp();
        asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
    }

    tc_fence_before();
    __syncthreads();
    if (*abort_flag) {  // a role gave up: loads and MMAs may be in flight
        if (threadIdx.x == 0) drain_ring<S>(full, max(begun_by[0], begun_by[1]), drain_limit(p));
        if (warp == 1 && elect_one()) {
            umma_commit(smem_u32(drain));
            mbar_drain(smem_u32(drain), 0u, drain_limit(p));
        }
    }
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(512u) : "memory");
    }
}

// ---- two CTAs per 256 x 192 tile (cta_group::2): large products
//
// Each CTA of a pair holds 128 rows of A and 96 of B, its half of the results (128
// rows x 192 columns) and the exponents of its rows of A and of all 192 of B: 28 KB of
// codes for 384 cycles of MMA, where a lone CTA would load 40. The even CTA's one
// thread issues the MMAs for both; loads of both CTAs complete on its barrier.
//
// 192 columns, because two accumulators of 256 leave no tensor memory for the
// exponents: sharing 64 columns between them made each span wait for the epilogue's
// first reads through two cluster-wide barriers, 0.8 us a span (8,192 x 8,192 x 4,096:
// 253 us). A tile starts in the middle of a 128-row group of exponents every other
// time; the MMA then takes them from two columns on.
//
// One warp loads A, another B (warp 2): a block's loads took one warp 340 cycles to
// issue. 12 epilogue warps (3-14) take 64
// columns each; a piece of 32 rows x 128 bytes leaves through a TMA store (store_piece
// where the result's rows are not 16-byte aligned). The odd CTA's epilogue warps free
// an accumulator on a barrier of their own, which the CTA's warp 1 passes on: an
// arrival on the other CTA's barrier is a release to the cluster, which waited 2,000
// cycles for a warp's stores.
//
// AST ("A stationary", rows of at most kAstBlocks blocks): a CTA takes consecutive
// tiles, keeps its 128 rows of A in shared memory while their row of tiles lasts, and
// streams only B: 12 KB a block instead of 28. L2 delivers about 61 bytes a cycle to an
// SM, less than 28 KB in a block's 384 cycles.

constexpr int kPairN = 192;
constexpr int kPairEpiWarps = 12;
constexpr int kPairThreads = 96 + 32 * kPairEpiWarps;
constexpr int kStages2 = 6;
constexpr int kTurnBytes2 = kPairEpiWarps * 32 * 128;
constexpr int kCodeTileB2 = kPairN / 2 * 128;
constexpr int kSf2 = 3 * kAtomBytes;
constexpr int kCodes2 = kCodeTile + kCodeTileB2;  // codes of one block
constexpr int kAstBlocks = 6;
constexpr int kSmem2 = 1024 + 256 + kTurnBytes2 + kStages2 * (kCodes2 + kSf2);
constexpr int kSmem2Ast = 1024 + 256 + kTurnBytes2 + kAstBlocks * kCodeTile + (kAstBlocks + 3) / 4 * kAtomBytes +
                          kStages2 * (kCodeTileB2 + 2 * kAtomBytes);
constexpr int kSfCols2 = 12;
constexpr int kSfBase2 = 2 * kPairN;
static_assert(kSmem2 <= 227 * 1024 && kSmem2Ast <= 227 * 1024 && kSfBase2 + kStages2 * kSfCols2 <= 512, "shared or tensor memory");

// The address of `addr` (this CTA's shared memory) in the pair's even CTA.
__device__ __forceinline__ uint32_t in_even_cta(uint32_t addr) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
    return r;
}

// A word written to the place of `p` in CTA `cta` of the pair.
__device__ __forceinline__ void store_cta(const volatile void* p, uint32_t cta, uint32_t value) {
    uint32_t at;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(tc::smem_u32(const_cast<const void*>(p))), "r"(cta));
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(value) : "memory");
}
__device__ __forceinline__ void store_even(const uint32_t* p, uint32_t value) { store_cta(p, 0u, value); }

// A load into this CTA's shared memory that completes on a barrier of the pair's even CTA.
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* tm, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
        "%3}], [%4];" ::"r"(dst),
        "l"((uint64_t)tm), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void arrive_remote(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Arrival on the same barrier of both CTAs once the MMAs issued so far are done.
__device__ __forceinline__ void commit_both(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
}

// store_piece through the TMA unit: the warp's turning buffer is its shared-memory box
// (32 rows x 128 bytes, 128-byte swizzle, which is the XOR of store_piece); rows past
// the result are left out by the tensor map. The store reads the buffer while the warp
// goes on; the next one waits for that.
__device__ __forceinline__ void store_tma(const uint32_t (&w)[32], uint8_t* buf, int lane, int row0, int col0,
                                          const CUtensorMap* tm) {
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i)
        *reinterpret_cast<uint4*>(buf + lane * 128 + ((i ^ (lane & 7)) << 4)) =
            make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (lane == 0) {
        asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                         (uint64_t)tm),
                     "r"(col0), "r"(row0), "r"(tc::smem_u32(buf))
                     : "memory");
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
}

template <int OB, bool AST>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    k_block8_matmul_pair(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                         const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB,
                         const __grid_constant__ CUtensorMap tmOut, const MmArgs p) {
    using namespace tc;
    constexpr int S = kStages2;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sA = smem;
    uint8_t* sB = sA + (AST ? kAstBlocks : S) * kCodeTile;
    uint8_t* turn = sB + S * kCodeTileB2;
    uint8_t* sSfA = turn + kTurnBytes2;  // exponents of A: a stage's, or (AST) the row of tiles'
    uint8_t* sSfB = sSfA + (AST ? (kAstBlocks + 3) / 4 : S) * kAtomBytes;
    uint64_t* bars = reinterpret_cast<uint64_t*>(sSfB + S * 2 * kAtomBytes);
    uint64_t* full = bars;            // (even CTA) both CTAs' loads of a stage
    uint64_t* empty = bars + S;       // (each CTA) the MMAs are done with a stage
    uint64_t* tfull = bars + 2 * S;   // (each CTA) an accumulator is complete
    uint64_t* tempty = tfull + 2;     // (each CTA) its epilogue has read an accumulator
    uint64_t* odd_empty = tfull + 4;  // (even CTA) so has the odd CTA's
    uint64_t* drain = tfull + 6;
    uint64_t* afull = tfull + 7;      // (AST; even CTA) both CTAs' rows of A
    uint64_t* aempty = tfull + 8;     // (AST; each CTA) the MMAs are done with them
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tfull + 9);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile int* other_abort = abort_flag + 1;  // the other CTA's, as it ended
    uint32_t* begun_by = tmem_slot + 3;          // (even CTA) stages, or rows of A, that each CTA's loaders began

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t rank;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    const int64_t tiles = (int64_t)p.m_tiles * p.n_tiles;
    // this pair's tiles: every step-th, or (AST) consecutive ones
    const int64_t pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    const int64_t first = AST ? pair * tiles / pairs : pair;
    const int64_t end = AST ? (pair + 1) * tiles / pairs : tiles;
    const int64_t step = AST ? 1 : pairs;
    const int groups = (p.nkb + 3) / 4;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(smem_u32(&full[s]), AST ? 1 : 2);  // a load of A, one of B
            mbar_init(smem_u32(&empty[s]), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(smem_u32(&tfull[a]), 1);
            mbar_init(smem_u32(&tempty[a]), kPairEpiWarps);
            mbar_init(smem_u32(&odd_empty[a]), 1);
        }
        mbar_init(smem_u32(drain), 1);
        mbar_init(smem_u32(afull), 1);
        mbar_init(smem_u32(aempty), 1);
        *abort_flag = *other_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(512u)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    pdl_wait();
    pdl_release();

    if (AST && warp == 0) {
        int last_m = -1;
        uint32_t rows = 0;  // rows of tiles begun
        bool ok = true;
        for (int64_t t = first; t < end && ok; t += step) {
            const int m = (int)(t / p.n_tiles);
            if (m == last_m) continue;
            last_m = m;
            ok = wait_bar<true>(smem_u32(aempty), (rows & 1u) ^ 1u, p.wait_limit, p.status, abort_flag);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            ++rows;
            if (elect_one()) {
                const int am = 2 * m + (int)rank;
                if (rank == 0) mbar_expect_tx(smem_u32(afull), (uint32_t)(2 * (p.nkb * kCodeTile + groups * kAtomBytes)));
                const uint32_t fb = in_even_cta(smem_u32(afull));
                for (int kb = 0; kb < p.nkb; ++kb) tma_load_pair(smem_u32(sA + kb * kCodeTile), &tmA, kb * kBlock, am * 128, fb);
                for (int g = 0; g < groups; ++g)
                    tma_load_pair(smem_u32(sSfA + g * kAtomBytes), &tmSA, 0, am * groups + g, fb);
            }
            __syncwarp();
        }
        if (lane == 0) store_even(&begun_by[2 * rank], rows);
    } else if (warp == 0 || warp == 2) {
        const bool loads_a = warp == 0;
        int stage = 0;
        uint32_t phase = 0, begun = 0;
        bool ok = true;
        for (int64_t t = first; t < end && ok; t += step) {
            const int m = (int)(t / p.n_tiles), n = (int)(t - (int64_t)m * p.n_tiles);
            const int am = 2 * m + (int)rank;  // this CTA's 128-row group of A
            const int sb = 3 * n / 2;          // the first 128-row group of the tile's rows of B
            for (int kb = 0; kb < p.nkb; ++kb) {
                ok = wait_warp<true>(smem_u32(&empty[stage]), phase ^ 1u, p.wait_limit, p.status, abort_flag);
                if (!ok) break;
                ++begun;
                if (elect_one()) {
                    uint8_t* sfb = sSfB + stage * 2 * kAtomBytes;
                    const uint32_t fb = in_even_cta(smem_u32(&full[stage]));
                    if (loads_a) {
                        if (rank == 0)
                            mbar_expect_tx(smem_u32(&full[stage]),
                                           (uint32_t)(2 * (kCodeTile + ((kb & 3) == 0 ? kAtomBytes : 0))));
                        tma_load_pair(smem_u32(sA + stage * kCodeTile), &tmA, kb * kBlock, am * 128, fb);
                        if ((kb & 3) == 0) tma_load_pair(smem_u32(sSfA + stage * kAtomBytes), &tmSA, 0, am * groups + (kb >> 2), fb);
                    } else {
                        if (rank == 0)
                            mbar_expect_tx(smem_u32(&full[stage]),
                                           (uint32_t)(2 * (kCodeTileB2 + ((kb & 3) == 0 ? 2 * kAtomBytes : 0))));
                        tma_load_pair(smem_u32(sB + stage * kCodeTileB2), &tmB, kb * kBlock,
                                      n * kPairN + (int)rank * (kPairN / 2), fb);
                        if ((kb & 3) == 0) {
                            tma_load_pair(smem_u32(sfb), &tmSB, 0, sb * groups + (kb >> 2), fb);
                            tma_load_pair(smem_u32(sfb + kAtomBytes), &tmSB, 0, (sb + 1) * groups + (kb >> 2), fb);
                        }
                    }
                }
                __syncwarp();
                if (++stage == S) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        if (lane == 0) store_even(&begun_by[2 * rank + (loads_a ? 0 : 1)], begun);
    } else if (warp == 1) {
        if (rank == 0) {
            int stage = 0, slot = S - 1;
            uint32_t phase = 0, span = 0;  // spans issued
            uint32_t rows = 0;             // (AST) rows of tiles begun
            int last_m = -1;
            bool ok = true;
            const uint64_t desc0 = smem_desc(0u, 2ull, 1024u);
            const uint32_t a_base = smem_u32(sA) >> 4, b_base = smem_u32(sB) >> 4;
            for (int64_t t = first; t < end && ok; t += step) {
                const int m = (int)(t / p.n_tiles), n = (int)(t - (int64_t)m * p.n_tiles);
                if (AST && m != last_m) {
                    last_m = m;
                    ok = wait_warp<true>(smem_u32(afull), rows & 1u, p.wait_limit, p.status, abort_flag);
                    ++rows;
                }
                // four blocks share a group of exponents; unrolled, so that what the MMAs
                // take but a block's stage is fixed
                for (int kb0 = 0; kb0 < p.nkb && ok; kb0 += 4) {
                    if (kb0 % kSpan == 0) {
                        const uint32_t parity = ((span >> 1) & 1u) ^ 1u;
                        ok = wait_warp<true>(smem_u32(&tempty[span & 1u]), parity, p.wait_limit, p.status, abort_flag) &&
                             wait_warp<true>(smem_u32(&odd_empty[span & 1u]), parity, p.wait_limit, p.status, abort_flag);
                    }
                    if (++slot == S) slot = 0;
                    const uint32_t sf = tmem_base + (uint32_t)(kSfBase2 + slot * kSfCols2);
                    const uint32_t sfb = sf + 4 + 2 * (n & 1);
                    const uint32_t acc = tmem_base + (span & 1u) * kPairN;
                    const int blocks = min(4, p.nkb - kb0);
                    const bool last = kb0 % kSpan + 4 == kSpan || kb0 + blocks == p.nkb;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (i >= blocks) break;
                        ok = ok && wait_warp<true>(smem_u32(&full[stage]), phase, p.wait_limit, p.status, abort_flag);
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t a_lo = a_base + (uint32_t)(AST ? kb0 + i : stage) * (kCodeTile >> 4);
                        const uint32_t b_lo = b_base + (uint32_t)stage * (kCodeTileB2 >> 4);
                        if (elect_one()) {
                            if (i == 0) {
                                copy_exponents<2>(sf, smem_u32(sSfA + (AST ? kb0 >> 2 : stage) * kAtomBytes));
                                copy_exponents<2>(sf + 4, smem_u32(sSfB + stage * 2 * kAtomBytes));
                                copy_exponents<2>(sf + 8, smem_u32(sSfB + (stage * 2 + 1) * kAtomBytes));
                            }
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                umma_block8<2>(acc, desc0 | (a_lo + 2 * kk), desc0 | (b_lo + 2 * kk),
                                               mm_idesc(256, kPairN, (uint32_t)i), sf, sfb,
                                               (i | kk) != 0 ? 1u : (uint32_t)(kb0 % kSpan));
                            commit_both(smem_u32(&empty[stage]));
                            if (last && i == blocks - 1) {
                                commit_both(smem_u32(&tfull[span & 1u]));
                                if (AST && kb0 + blocks == p.nkb && (t + 1 == end || n == p.n_tiles - 1))
                                    commit_both(smem_u32(aempty));
                            }
                        }
                        __syncwarp();
                        if (++stage == S) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                    if (last) ++span;
                }
            }
        } else if (lane == 0) {
            const int64_t spans = first < end ? (end - first + step - 1) / step * ((p.nkb + kSpan - 1) / kSpan) : 0;
            for (int64_t i = 0; i < spans; ++i) {
                if (!wait_bar(smem_u32(&tempty[i & 1]), (uint32_t)(i >> 1) & 1u, p.wait_limit, p.status, abort_flag)) break;
                arrive_remote(in_even_cta(smem_u32(&odd_empty[i & 1])));
            }
        }
    } else {
        const int ew = warp - 3;
        const int q = warp & 3, third = ew >> 2;
        const uint32_t lane_base = (uint32_t)(32 * q) << 16;
        uint8_t* buf = turn + ew * 32 * 128;
        uint32_t span = 0;
        bool ok = true;
        for (int64_t t = first; t < end && ok; t += step) {
            const int m = (int)(t / p.n_tiles), n = (int)(t - (int64_t)m * p.n_tiles);
            const int64_t row0 = (int64_t)m * 256 + rank * 128 + 32 * q;
            const int64_t col0 = (int64_t)n * kPairN + third * 64;
            uint32_t sum[2][32];
            clear_sums(sum);
            for (int kb = 0; kb < p.nkb; kb += kSpan) {
                const uint32_t acc = span & 1u;
                if (!wait_warp<true>(smem_u32(&tfull[acc]), (span >> 1) & 1u, p.wait_limit, p.status, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t tbase = tmem_base + lane_base + acc * kPairN + (uint32_t)(third * 64);
#pragma unroll
                for (int i = 0; i < 2; ++i) add_columns(tbase + 32 * i, sum[i]);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&tempty[acc]));
                ++span;
            }
            if (!ok) break;
            if (row0 >= p.m_rows) continue;
            if (p.vec_ok && col0 + 64 <= p.n_rows) {
                if (OB == 4) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) store_tma(sum[i], buf, lane, (int)row0, (int)col0 + 32 * i, &tmOut);
                } else {
                    uint32_t w[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        w[e] = pack_out(sum[e >> 4][2 * (e & 15)], sum[e >> 4][2 * (e & 15) + 1], p.bf16);
                    store_tma(w, buf, lane, (int)row0, (int)col0, &tmOut);
                }
            } else {  // (a TMA store would fill the last 16 bytes of a row)
                if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                store_rows<OB, 2>(sum, buf, lane, row0, col0, p);
            }
        }
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }

    tc_fence_before();
    __syncthreads();
    // neither CTA's shared or tensor memory goes while the other may still use it, nor
    // while loads or MMAs of a pair that gave up may be in flight (the even CTA's barriers
    // stand for both CTAs' loads)
    if (threadIdx.x == 0 && *abort_flag) store_cta(other_abort, rank ^ 1u, 1u);
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (*abort_flag || *other_abort) {
        if (rank == 0 && threadIdx.x == 0) {
            const uint32_t a = max(begun_by[0], begun_by[2]), b = max(begun_by[1], begun_by[3]);
            drain_ring<S>(full, AST ? b : max(a, b), drain_limit(p));
            if (AST && a > 0) mbar_drain(smem_u32(afull), (a - 1) & 1u, drain_limit(p));
        }
        if (rank == 0 && warp == 1 && elect_one()) {
            asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                             smem_u32(drain))
                         : "memory");
            mbar_drain(smem_u32(drain), 0u, drain_limit(p));
        }
        __syncwarp();
        asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(512u) : "memory");
    }
}

}  // namespace b8
}  // namespace em
