// Matrices in block-scaled 4-bit floating point: layout, quantisation, reading back.
//
// Bound by memory: 2 bytes an element in and 0.53 to 0.56 out (quantising), or the reverse. A lane has 16 consecutive values of a row at a time,
// 32 bytes in one load where they are aligned: a warp reads whole lines (with 64 bytes a lane in four loads, each touched a quarter of twice as many
// lines: 89 us for 4001 x 11008 and back, now 49), and a scale needs no more than one other lane. A row has as many warps as keep all of it in registers (up to
// 16384 columns), so that blocks of 16, whose scales depend on the row's largest element, read it once.
// The 8 rows of a CTA are the pairs (2p, 2p + 1) of each 32 of a tile's 128, so that the two halves of a 32-byte sector of codes, and the
// eight words of a sector of scales, are written by one CTA at about the same time.
//
// The quotients. x has 11 significant bits, a scale 4, a midpoint between two codes 3: a quotient x / scale is a midpoint or at least 2^-11
// of one away, so that a binary32 quotient which is exact where it has few bits rounds as the true one does. It is formed by a
// reciprocal and one Newton correction of the quotient, q + (x - q s) / s, whose remainder is exact, without a division for each element.
// The same holds for m / 6 and e4m3.
#include "fp4_common.cuh"

namespace sgemv {

namespace {

constexpr int kWarpsQ = 8;

constexpr int kHeld = 4;  // pieces of 16 values that a lane keeps

struct QuantParams {
    Fp4Matrix m;
    const void* x;   // or the output of read
    int64_t stride;
    int32_t* status;
    int wpr;         // warps a row
    int lanes;       // lanes a row, where rows are short
    int align;       // of the rows' pieces: 32 bytes, 16, or 0 (an element)
};

__device__ __forceinline__ float reciprocal(float x) {  // to a unit in the last place or so
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The row of a CTA's slot.
__device__ __forceinline__ int row_of_slot(const Fp4Matrix& m, int64_t slot) {
    if (m.tile < 128) return static_cast<int>(slot);
    const int s = static_cast<int>(slot & 127);
    return static_cast<int>(slot - s) + 32 * ((s >> 1) & 3) + 2 * (s >> 3) + (s & 1);
}

// 16 values of a row from column 16 c, zeros past its end.
template <typename T>
__device__ __forceinline__ void load16(const T* row, int c, int k, int align, uint32_t (&w)[8]) {
    if (align == 32 && 16 * c < k) {
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                     : "l"(row + 16 * c));
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (16 * c + 8 * i < k) v = *reinterpret_cast<const uint4*>(row + 16 * c + 8 * i);
            w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
        }
    }
}
// Rows that start anywhere go through shared memory, so that a warp reads and writes whole words next to one another: the 512 values from column
// 16 * base on as 257 words, a word of two halves of which one lies outside of the row by halves.
struct Line {
    const unsigned short* at;  // the first value
    int n;                     // values
    bool odd;                  // it is the upper half of a word
    template <typename T>
    __device__ __forceinline__ Line(const T* row, int base, int k)
        : at(reinterpret_cast<const unsigned short*>(row) + 16ll * base), n(min(512, k - 16 * base)), odd((reinterpret_cast<uintptr_t>(row) & 2) != 0) {}
};
__device__ __forceinline__ void load_line(const Line& l, int lane, uint32_t (&v)[9]) {
#pragma unroll
    for (int i = 0; i < 9; ++i) {
        const int first = 2 * (lane + 32 * i) - l.odd;  // of the word's two values
        v[i] = 0;
        if (first >= 0 && first + 1 < l.n) {
            v[i] = *reinterpret_cast<const uint32_t*>(l.at + first);
        } else {
            if (first >= 0 && first < l.n) v[i] = l.at[first];
            if (first + 1 >= 0 && first + 1 < l.n) v[i] |= static_cast<uint32_t>(l.at[first + 1]) << 16;
        }
    }
}
__device__ __forceinline__ void spread_line(const Line& l, int lane, const uint32_t (&v)[9], uint32_t* buf, uint32_t (&w)[8]) {
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 9; ++i)
        if (i < 8 || lane == 0) buf[lane + 32 * i] = v[i];
    __syncwarp();
    const uint4 a = *reinterpret_cast<const uint4*>(buf + 8 * lane), b = *reinterpret_cast<const uint4*>(buf + 8 * lane + 4);
    const uint32_t u[9] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, buf[8 * lane + 8]};
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = l.odd ? __funnelshift_r(u[i], u[i + 1], 16) : u[i];
}
// The largest magnitude of 8 words' elements, as 16 bits (infinities and NaN above all numbers).
__device__ __forceinline__ uint32_t most16(const uint32_t (&w)[8]) {
    uint32_t m = w[0] & 0x7FFF7FFFu;
#pragma unroll
    for (int i = 1; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
    return max(m & 0xFFFFu, m >> 16);
}
template <typename T>
__device__ __forceinline__ float as_f32(uint32_t bits) {
    return two_f32<T>(bits).x;
}
template <typename T>
constexpr uint32_t kInfBits = 0x7C00u;
template <>
constexpr uint32_t kInfBits<__nv_bfloat16> = 0x7F80u;

// Codes of 16 values whose block's largest magnitude is `most` (as 16 bits), and the block's scale. unit and down: the row's power of two and its inverse.
template <typename T, int kBlock>
__device__ __forceinline__ uint2 encode16(const uint32_t (&w)[8], uint32_t most, float unit, float down, uint32_t& scale) {
    float s, inv;
    if constexpr (kBlock == 32) {
        scale = max(0, static_cast<int>(__float_as_uint(as_f32<T>(most)) >> 23) - 2);
        inv = __uint_as_float((254u - scale) << 23), s = 0.0f;
    } else {
        const float m = as_f32<T>(most) * down, sixth = m * (1.0f / 6.0f);
        scale = to_e4m3(fmaf(fmaf(-6.0f, sixth, m), 1.0f / 6.0f, sixth));
        s = from_e4m3(scale) * unit;
        inv = s > 0.0f ? reciprocal(s) : 0.0f;
    }
    uint32_t codes[2];
    const uint64_t r = pair(inv, inv), d = pair(-s, -s);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float t[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = two_f32<T>(w[4 * i + j]);
            const uint64_t v = pair(f.x, f.y);
            uint64_t q = mul2(v, r);
            if constexpr (kBlock == 16) q = fma2(fma2(q, d, v), r, q);
            const float2 g = parts_of(q);
            t[2 * j] = g.x, t[2 * j + 1] = g.y;
        }
        codes[i] = to_e2m1x8(t);
    }
    return make_uint2(codes[0], codes[1]);
}
// The row's power of two for its largest magnitude (1 for a row with none, or with an element that is no number), and its inverse. 2688 = 1.3125 * 2^11
template <typename T>
__device__ __forceinline__ void row_unit(uint32_t most, float& unit, float& down) {
    const uint32_t b = __float_as_uint(as_f32<T>(most));
    const int e = most >= kInfBits<T> || b == 0 ? 0 : max(-100, static_cast<int>(b >> 23) - 138 + ((b & 0x7FFFFFu) > 0x280000u));
    unit = __uint_as_float(static_cast<uint32_t>(127 + e) << 23), down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
}

template <typename T, int kBlock>
__global__ void __launch_bounds__(32 * kWarpsQ) quantize_kernel(const QuantParams p) {
    __shared__ uint32_t s_most[kWarpsQ];
    __shared__ __align__(16) uint32_t s_line[kWarpsQ][260];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int slot = warp / p.wpr, part = warp % p.wpr;
    if (threadIdx.x < kWarpsQ) s_most[threadIdx.x] = 0;
    pdl_launch_dependents();
    const int row = row_of_slot(p.m, static_cast<int64_t>(blockIdx.x) * (kWarpsQ / p.wpr) + slot);
    const bool live = row < p.m.rows;
    const T* const x = static_cast<const T*>(p.x) + (live ? row : 0) * p.stride;
    const int pieces = live ? p.m.kp / 16 : 0, step = 32 * p.wpr, first = 32 * part + lane;
    __syncthreads();
    pdl_wait();
    uint32_t held[kHeld][8];
    uint32_t held_most[kHeld];
    const auto some = [&](int i) { return 32 * part + i * step < pieces; };  // whether any lane of the warp has its piece i
    if (p.align > 0) {
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const int c = first + i * step;
#pragma unroll
            for (int e = 0; e < 8; ++e) held[i][e] = 0;
            if (c < pieces) load16(x, c, p.m.k, p.align, held[i]);
        }
    } else {
        uint32_t v[kHeld][9];
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
            if (some(i)) load_line(Line(x, 32 * part + i * step, p.m.k), lane, v[i]);
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
            if (some(i)) spread_line(Line(x, 32 * part + i * step, p.m.k), lane, v[i], s_line[warp], held[i]);
    }
#pragma unroll
    for (int i = 0; i < kHeld; ++i) held_most[i] = some(i) ? most16(held[i]) : 0;
    const auto load = [&](int base, uint32_t (&w)[8]) {  // piece base + lane of a long row
        if (p.align > 0) {
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = 0;
            if (base + lane < pieces) load16(x, base + lane, p.m.k, p.align, w);
        } else {
            const Line l(x, base, p.m.k);
            uint32_t v[9];
            load_line(l, lane, v);
            spread_line(l, lane, v, s_line[warp], w);
        }
    };
    float unit = 1.0f, down = 1.0f;
    bool bad = false;
    if constexpr (kBlock == 16) {
        // the row's largest magnitude, and from it the row's power of two
        uint32_t most = max(max(held_most[0], held_most[1]), max(held_most[2], held_most[3]));
        for (int base = 32 * part + kHeld * step; base < pieces; base += step) {
            uint32_t w[8];
            load(base, w);
            most = max(most, most16(w));
        }
        most = __reduce_max_sync(0xFFFFFFFFu, most);
        if (p.wpr > 1) {
            if (lane == 0) atomicMax(&s_most[slot], most);
            __syncthreads();
            most = s_most[slot];
        }
        bad = most >= kInfBits<T>;
        row_unit<T>(most, unit, down);
    }
    uint32_t seen = 0;
    uint8_t* const row_codes = codes_at(p.m, live ? row : 0, 0) + 8 * (lane & 1);
    uint8_t* const row_scales = scales_at(p.m, live ? row : 0, 0);
    const int chunk_bytes = p.m.tile * 16;
    // Piece c of the row, by the whole warp (lanes past the row's end have zeros).
    const auto quantize = [&](int c, const uint32_t (&w)[8], uint32_t most) {
        if constexpr (kBlock == 32) {
            most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
            seen = max(seen, most);
        }
        uint32_t scale;
        const uint2 codes = encode16<T, kBlock>(w, most, unit, down, scale);
        // four scales a word: of 4 lanes, or of every second of 8
        constexpr int kApart = kBlock / 16;
        if (c >= pieces) scale = 0;
        scale |= __shfl_down_sync(0xFFFFFFFFu, scale, kApart) << 8;
        scale |= __shfl_down_sync(0xFFFFFFFFu, scale, 2 * kApart) << 16;
        if (c < pieces) {
            *reinterpret_cast<uint2*>(row_codes + static_cast<int64_t>(c / 2) * chunk_bytes) = codes;
            if (lane % (4 * kApart) == 0) *reinterpret_cast<uint32_t*>(row_scales + static_cast<int64_t>(c / (4 * kApart)) * 512) = scale;
        }
    };
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
        if (some(i)) quantize(first + i * step, held[i], held_most[i]);
    for (int base = 32 * part + kHeld * step; base < pieces; base += step) {
        uint32_t w[8];
        load(base, w);
        quantize(base + lane, w, most16(w));
    }
    if constexpr (kBlock == 32) {
        seen = __reduce_max_sync(0xFFFFFFFFu, seen);
        if (p.wpr > 1) {
            if (lane == 0) atomicMax(&s_most[slot], seen);
            __syncthreads();
            seen = s_most[slot];
        }
        bad = seen >= kInfBits<T>;
    }
    if (bad) {  // zeros over what this lane wrote (a block of 32 is written before its row is known to hold no numbers)
#pragma unroll 1
        for (int c = first; c < pieces; c += step) {
            *reinterpret_cast<uint2*>(row_codes + static_cast<int64_t>(c / 2) * chunk_bytes) = make_uint2(0, 0);
            if (lane % (kBlock / 4) == 0) *reinterpret_cast<uint32_t*>(row_scales + static_cast<int64_t>(c / (kBlock / 4)) * 512) = 0;
        }
    }
    if (live && part == 0 && lane == 0) {
        p.m.row_scale[row] = bad ? __int_as_float(0x7FC00000) : unit;
        if (bad) report(p.status, SGEMV_ERR_NONFINITE);
    }
}

// The n values (512 at most) in buf, to where a row starts or 16 values further, by the warp: as words next to one another.
template <typename T>
__device__ __forceinline__ void store_words(T* at, int n, int lane, const uint32_t* buf) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll 4
        for (int i = lane; i < n; i += 32) reinterpret_cast<uint32_t*>(at)[i] = buf[i];
    } else {
        const bool odd = (reinterpret_cast<uintptr_t>(at) & 2) != 0;
        unsigned short* const h = reinterpret_cast<unsigned short*>(at);
#pragma unroll
        for (int i = 0; i < 9; ++i) {
            const int word = lane + 32 * i, first = 2 * word - odd;
            if (first >= n) break;
            const uint32_t here = word < 256 ? buf[word] : 0, before = odd && word > 0 ? buf[word - 1] : 0;
            const uint32_t v = odd ? __funnelshift_r(before, here, 16) : here;
            if (first >= 0 && first + 1 < n) {
                *reinterpret_cast<uint32_t*>(h + first) = v;
            } else {
                if (first >= 0) h[first] = static_cast<unsigned short>(v);
                if (first + 1 >= 0 && first + 1 < n) h[first + 1] = static_cast<unsigned short>(v >> 16);
            }
        }
    }
}
// The warp's 512 values from column 16 * base on, 16 a lane.
template <typename T>
__device__ __forceinline__ void store_line(T* row, int base, int k, int lane, const uint32_t (&w)[8 * sizeof(T) / 2], uint32_t* buf) {
    constexpr int kWords = 8 * sizeof(T) / 2;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kWords; i += 4) *reinterpret_cast<uint4*>(buf + kWords * lane + i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
    __syncwarp();
    store_words(row + 16ll * base, min(512, k - 16 * base), lane, buf);
}

// The 16 values of 8 bytes of codes.
template <int kBlock>
__device__ __forceinline__ void decode16(const uint8_t* at, uint32_t scale, float unit, float (&f)[16]) {
    const uint2 codes = *reinterpret_cast<const uint2*>(at);
    const float s = (kBlock == 16 ? from_e4m3(scale) : from_e8m0(scale)) * unit;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t h[4];
        from_e2m1x8(i ? codes.y : codes.x, h);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 v = two_f32<__half>(h[j]);
            f[8 * i + 2 * j] = v.x * s, f[8 * i + 2 * j + 1] = v.y * s;
        }
    }
}
template <typename T>
__device__ __forceinline__ void to_words(const float (&f)[16], uint32_t (&w)[8 * sizeof(T) / 2]) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(8 * sizeof(T) / 2); ++i) {
        if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(f[i]);
        else w[i] = pack_two<T>(f[2 * i], f[2 * i + 1]);
    }
}
// The first n of a lane's 16 values, to an address of the alignment `align` (32 or 16 bytes).
template <typename T>
__device__ __forceinline__ void store16(T* to, int n, int align, const float (&f)[16], const uint32_t (&w)[8 * sizeof(T) / 2]) {
    if (n >= 16) {
#pragma unroll
        for (int i = 0; i < static_cast<int>(8 * sizeof(T) / 2); i += 8) {
            if (align == 32) {
                asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(reinterpret_cast<uint32_t*>(to) + i), "r"(w[i]), "r"(w[i + 1]),
                             "r"(w[i + 2]), "r"(w[i + 3]), "r"(w[i + 4]), "r"(w[i + 5]), "r"(w[i + 6]), "r"(w[i + 7])
                             : "memory");
            } else {
                reinterpret_cast<uint4*>(to)[i / 4] = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
                reinterpret_cast<uint4*>(to)[i / 4 + 1] = make_uint4(w[i + 4], w[i + 5], w[i + 6], w[i + 7]);
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < 16; ++j)
            if (j < n) to[j] = from_f32<T>(f[j]);
    }
}

template <typename T, int kBlock>
__global__ void __launch_bounds__(32 * kWarpsQ) read_kernel(const QuantParams p) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int slot = warp / p.wpr, part = warp % p.wpr;
    pdl_launch_dependents();
    const int row = row_of_slot(p.m, static_cast<int64_t>(blockIdx.x) * (kWarpsQ / p.wpr) + slot);
    pdl_wait();
    if (row >= p.m.rows) return;
    T* const out = const_cast<T*>(static_cast<const T*>(p.x)) + row * p.stride;
    const float unit = p.m.row_scale[row];
    const uint8_t *const row_codes = codes_at(p.m, row, 0), *const row_scales = scales_at(p.m, row, 0);
    const int chunk_bytes = p.m.tile * 16;
    __shared__ __align__(16) uint32_t s_line[kWarpsQ][32 * 8 * sizeof(T) / 2];
    for (int base = 32 * part; 16 * base < p.m.k; base += 32 * p.wpr) {
        const int c = base + lane;
        const int at = min(c, p.m.kp / 16 - 1);  // (a lane without a piece among others that have one: any)
        float f[16];
        decode16<kBlock>(row_codes + static_cast<int64_t>(at / 2) * chunk_bytes + 8 * (at & 1),
                         row_scales[static_cast<int64_t>(at * 16 / kBlock / 4) * 512 + at * 16 / kBlock % 4], unit, f);
        constexpr int kWords = 8 * sizeof(T) / 2;  // of 16 values
        uint32_t w[kWords];
        to_words<T>(f, w);
        T* const to = out + 16 * c;
        if (p.align == 0) {
            store_line(out, base, p.m.k, lane, w, s_line[warp]);
        } else {
            store16(to, p.m.k - 16 * c, p.align, f, w);
        }
    }
}

// Short rows: p.lanes lanes a row (8 or 16), a piece each, so that a warp has 4 or 2 rows (328153 rows of 122 values: 158 us with a warp a row, 29 so).
// 16 values that start anywhere are read by the lane itself: neighbours' words are in the same lines, which L1 holds.
template <typename T, int kBlock>
__global__ void __launch_bounds__(32 * kWarpsQ) quantize_short_kernel(const QuantParams p) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = lane % p.lanes;
    pdl_launch_dependents();
    const int64_t slot = (static_cast<int64_t>(blockIdx.x) * kWarpsQ + warp) * (32 / p.lanes) + lane / p.lanes;
    const bool live = slot < p.m.rows, mine = live && c < p.m.kp / 16;
    const int row = live ? static_cast<int>(slot) : 0;
    const T* const x = static_cast<const T*>(p.x) + row * p.stride;
    pdl_wait();
    uint32_t w[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (mine) {
        if (p.align > 0) {
            load16(x, c, p.m.k, p.align, w);
        } else {
            const Line l(x, c, p.m.k);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (!l.odd && 2 * i + 1 < l.n) {
                    w[i] = *reinterpret_cast<const uint32_t*>(l.at + 2 * i);
                } else {
                    if (2 * i < l.n) w[i] = l.at[2 * i];
                    if (2 * i + 1 < l.n) w[i] |= static_cast<uint32_t>(l.at[2 * i + 1]) << 16;
                }
            }
        }
    }
    uint32_t most = most16(w), row_most = most;
    for (int d = p.lanes / 2; d > 0; d >>= 1) row_most = max(row_most, __shfl_xor_sync(0xFFFFFFFFu, row_most, d));
    if constexpr (kBlock == 32) most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
    float unit = 1.0f, down = 1.0f;
    if constexpr (kBlock == 16) row_unit<T>(row_most, unit, down);
    uint32_t scale;
    uint2 codes = encode16<T, kBlock>(w, most, unit, down, scale);
    constexpr int kApart = kBlock / 16;
    const bool bad = row_most >= kInfBits<T>;
    if (bad) codes = make_uint2(0, 0);
    if (bad || !mine) scale = 0;
    scale |= __shfl_down_sync(0xFFFFFFFFu, scale, kApart) << 8;
    scale |= __shfl_down_sync(0xFFFFFFFFu, scale, 2 * kApart) << 16;
    if (mine) {
        *reinterpret_cast<uint2*>(codes_at(p.m, row, c / 2) + 8 * (c & 1)) = codes;
        if (c % (4 * kApart) == 0) *reinterpret_cast<uint32_t*>(scales_at(p.m, row, c / (4 * kApart))) = scale;
    }
    if (live && c == 0) {
        p.m.row_scale[row] = bad ? __int_as_float(0x7FC00000) : unit;
        if (bad) report(p.status, SGEMV_ERR_NONFINITE);
    }
}

// The same way back (328153 rows of 122 values: 95 us with a warp a row, 42 so).
template <typename T, int kBlock>
__global__ void __launch_bounds__(32 * kWarpsQ) read_short_kernel(const QuantParams p) {
    constexpr int kWords = 8 * sizeof(T) / 2;
    __shared__ __align__(16) uint32_t s_line[kWarpsQ][32 * kWords + 4];  // (the word behind a row, whose value is not used, may be behind the last)
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = lane % p.lanes;
    pdl_launch_dependents();
    const int64_t base = (static_cast<int64_t>(blockIdx.x) * kWarpsQ + warp) * (32 / p.lanes);  // the warp's first row
    const int64_t slot = base + lane / p.lanes;
    pdl_wait();
    uint32_t w[kWords] = {};
    if (slot < p.m.rows && 16 * c < p.m.k) {
        const int row = static_cast<int>(slot);
        float f[16];
        decode16<kBlock>(codes_at(p.m, row, c / 2) + 8 * (c & 1), scales_at(p.m, row, c * 16 / kBlock / 4)[c * 16 / kBlock % 4], p.m.row_scale[row], f);
        to_words<T>(f, w);
        if (p.align > 0) store16(const_cast<T*>(static_cast<const T*>(p.x)) + row * p.stride + 16 * c, p.m.k - 16 * c, p.align, f, w);
    }
    if (p.align > 0) return;
    // rows that start anywhere: by the whole warp, a row after the other
    uint32_t* const buf = s_line[warp];
#pragma unroll
    for (int i = 0; i < kWords; i += 4) *reinterpret_cast<uint4*>(buf + kWords * lane + i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
    __syncwarp();
    for (int r = 0; r < 32 / p.lanes && base + r < p.m.rows; ++r)
        store_words(const_cast<T*>(static_cast<const T*>(p.x)) + (base + r) * p.stride, p.m.k, lane, buf + r * p.lanes * kWords);
}

// Rows in pieces of 16 values: how the pieces are aligned.
int row_align(const void* p, int64_t stride, int rows, int k, int size) {
    if (is_aligned(p, 32) && k % 16 == 0 && (rows < 2 || stride * size % 32 == 0)) return 32;
    return is_aligned(p, 16) && k % 8 == 0 && (rows < 2 || stride * size % 16 == 0) ? 16 : 0;
}

// Warps a row: as few as hold it in registers; more, where rows are too few for 8 warps an SM, as far as each has 512 columns.
int warps_a_row(int rows, int k, int sms) {
    int w = 1;
    while (w < kWarpsQ && (k > 512 * kHeld * w || (static_cast<int64_t>(rows) * w < 8ll * sms && k > 512 * w))) w *= 2;
    return w;
}

int launch_rows(const sgemv_fp4_layout& l, QuantParams& p, void (*kern)(const QuantParams), void* stream) {
    DeviceInfo di;
    const int rc = device_info(&di);
    if (rc != SGEMV_OK) return rc;
    p.wpr = warps_a_row(l.rows, l.k, di.sm_count);
    const int64_t slots = (static_cast<int64_t>(l.rows) + l.tile - 1) / l.tile * l.tile;
    const int64_t used = l.tile < 128 ? l.rows : slots;
    const int64_t per = kWarpsQ / p.wpr;
    const cudaError_t e = launch_pdl(kern, dim3(static_cast<unsigned>((used + per - 1) / per)), dim3(32 * kWarpsQ), 0,
                                     static_cast<cudaStream_t>(stream), p);
    return e == cudaSuccess ? SGEMV_OK : SGEMV_ERR_CUDA;
}

// Rows that leave half of a warp's lanes, or more, without a piece; from the tiles of 128 rows on (below, both
// are one wave of the GPU: 2.0 to 2.6 us for 64 rows and for 65).
bool short_rows(const sgemv_fp4_layout& l) { return l.kp <= 256 && l.tile == 128; }

int launch_short(const sgemv_fp4_layout& l, QuantParams& p, void (*kern)(const QuantParams), void* stream) {
    DeviceInfo di;
    const int rc = device_info(&di);
    if (rc != SGEMV_OK) return rc;
    p.lanes = l.kp <= 128 ? 8 : 16;
    const int per = kWarpsQ * 32 / p.lanes;
    const cudaError_t e =
        launch_pdl(kern, dim3(static_cast<unsigned>((l.rows + per - 1) / per)), dim3(32 * kWarpsQ), 0, static_cast<cudaStream_t>(stream), p);
    return e == cudaSuccess ? SGEMV_OK : SGEMV_ERR_CUDA;
}

}  // namespace

int check_fp4_layout(const sgemv_fp4_layout* layout) {
    if (layout == nullptr) return SGEMV_ERR_ARG;
    sgemv_fp4_layout ref;
    if (sgemv_fp4_layout_query(layout->rows, layout->k, layout->block, &ref) != SGEMV_OK) return SGEMV_ERR_FORMAT;
    return ref.tile == layout->tile && ref.kp == layout->kp && ref.scale_off == layout->scale_off && ref.row_off == layout->row_off &&
                   ref.total_bytes == layout->total_bytes
               ? SGEMV_OK
               : SGEMV_ERR_FORMAT;
}

}  // namespace sgemv

using namespace sgemv;

extern "C" int sgemv_fp4_layout_query(int rows, int k, int block, sgemv_fp4_layout* out) {
    if (out == nullptr) return SGEMV_ERR_ARG;
    if (rows < 0 || rows > (1 << 24) || k < 1 || k > (1 << 20) || (block != 16 && block != 32)) return SGEMV_ERR_SHAPE;
    sgemv_fp4_layout l = {};
    l.rows = rows, l.k = k, l.block = block;
    l.tile = 8;
    while (l.tile < rows && l.tile < 128) l.tile *= 2;
    l.kp = (k + 63) / 64 * 64;
    const uint64_t tiles = (static_cast<uint64_t>(rows) + l.tile - 1) / l.tile, big = (static_cast<uint64_t>(rows) + 127) / 128;
    l.scale_off = tiles * l.tile * (l.kp / 2);
    l.row_off = l.scale_off + big * ((l.kp + 4 * block - 1) / (4 * block)) * 512;
    l.total_bytes = l.row_off + big * 512;
    *out = l;
    return SGEMV_OK;
}

extern "C" int sgemv_fp4_quantize(const sgemv_fp4_layout* layout, const void* x_dev, int dtype, int64_t stride, void* packed_dev,
                                  int32_t* status_dev, void* stream) {
    const int rc = check_fp4_layout(layout);
    if (rc != SGEMV_OK) return rc;
    if (dtype != SGEMV_F16 && dtype != SGEMV_BF16) return SGEMV_ERR_ARG;
    if (layout->rows == 0) return SGEMV_OK;
    if (x_dev == nullptr || packed_dev == nullptr) return SGEMV_ERR_ARG;
    if (layout->rows > 1 && (stride < layout->k || stride > (1ll << 40))) return SGEMV_ERR_ARG;
    if (!is_aligned(packed_dev, 16) || !is_aligned(x_dev, 2) || !is_aligned(status_dev, 4)) return SGEMV_ERR_ALIGN;
    const int64_t st = layout->rows > 1 ? stride : layout->k;
    const Bytes x(x_dev, 2 * ((layout->rows - 1) * st + layout->k));
    const Bytes written[] = {{packed_dev, layout->total_bytes}, {status_dev, 4}};
    if (!apart(written, {x})) return SGEMV_ERR_ARG;
    QuantParams p;
    p.m = Fp4Matrix(*layout, packed_dev);
    p.x = x_dev, p.stride = st, p.status = status_dev;
    p.align = row_align(x_dev, st, layout->rows, layout->k, 2);
    const bool half = dtype == SGEMV_F16;
    if (short_rows(*layout))
        return launch_short(*layout, p,
                            layout->block == 16 ? (half ? quantize_short_kernel<__half, 16> : quantize_short_kernel<__nv_bfloat16, 16>)
                                                : (half ? quantize_short_kernel<__half, 32> : quantize_short_kernel<__nv_bfloat16, 32>),
                            stream);
    return launch_rows(*layout, p,
                       layout->block == 16 ? (half ? quantize_kernel<__half, 16> : quantize_kernel<__nv_bfloat16, 16>)
                                           : (half ? quantize_kernel<__half, 32> : quantize_kernel<__nv_bfloat16, 32>),
                       stream);
}

extern "C" int sgemv_fp4_read(const sgemv_fp4_layout* layout, const void* packed_dev, void* out_dev, int dtype, int64_t stride,
                              void* stream) {
    const int rc = check_fp4_layout(layout);
    if (rc != SGEMV_OK) return rc;
    if (dtype < SGEMV_F16 || dtype > SGEMV_F32) return SGEMV_ERR_ARG;
    if (layout->rows == 0) return SGEMV_OK;
    if (out_dev == nullptr || packed_dev == nullptr) return SGEMV_ERR_ARG;
    if (layout->rows > 1 && (stride < layout->k || stride > (1ll << 40))) return SGEMV_ERR_ARG;
    const unsigned size = dtype == SGEMV_F32 ? 4 : 2;
    if (!is_aligned(packed_dev, 16) || !is_aligned(out_dev, size)) return SGEMV_ERR_ALIGN;
    const int64_t st = layout->rows > 1 ? stride : layout->k;
    if (rows_meet({out_dev, size * static_cast<uint64_t>(layout->k)}, layout->rows, size * st, {packed_dev, layout->total_bytes}))
        return SGEMV_ERR_ARG;
    QuantParams p;
    p.m = Fp4Matrix(*layout, packed_dev);
    p.x = out_dev, p.stride = st, p.status = nullptr;
    p.align = row_align(out_dev, st, layout->rows, layout->k, static_cast<int>(size));
    const bool b16 = layout->block == 16;
    if (short_rows(*layout))
        return launch_short(*layout, p,
                            dtype == SGEMV_F16    ? (b16 ? read_short_kernel<__half, 16> : read_short_kernel<__half, 32>)
                            : dtype == SGEMV_BF16 ? (b16 ? read_short_kernel<__nv_bfloat16, 16> : read_short_kernel<__nv_bfloat16, 32>)
                                                  : (b16 ? read_short_kernel<float, 16> : read_short_kernel<float, 32>),
                            stream);
    return launch_rows(*layout, p,
                       dtype == SGEMV_F16    ? (b16 ? read_kernel<__half, 16> : read_kernel<__half, 32>)
                       : dtype == SGEMV_BF16 ? (b16 ? read_kernel<__nv_bfloat16, 16> : read_kernel<__nv_bfloat16, 32>)
                                             : (b16 ? read_kernel<float, 16> : read_kernel<float, 32>),
                       stream);
}
