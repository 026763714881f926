// kv_rotate, kv_rotate_write, kv_rotate_write_q4: heads rotated by their tokens' positions, and the new tokens' keys and values
// appended to the pages with the rotation (and the rounding to 4 bits) on the way.
//
// A pair (a, b) of a head becomes m (a cos t - b sin t, a sin t + b cos t), t = position * frequency.  Frequencies are 64-bit
// fractions of a turn, so position * frequency is an integer product whose overflow drops whole turns: the angle of position
// 2^31 is as good as that of position 1 (in 32-bit floating point t is off by 0.06 at a million).
//
// 4-bit codes must not depend on how the angle was rounded: a border between two codes is 2^-5 of a value wide in steps of
// bf16, so one in 2^20 elements would come out otherwise than from exact angles.  Cosines and sines are therefore held in two
// floats (what is left is below 2^-37), the products keep what their rounding leaves (Dekker; Knuth's sum), and the result is rounded
// once to 32 bits and once to the element type, as a 16-bit cache would hold it, before it is rounded to 4 bits.
//
// Bound by bandwidth: every element is read and written once.  A CTA takes tokens one after another, a thread the same two pieces of
// 16 bytes of each, so that where they come from and go to is worked out once.  While a token's heads are turned, the next one's
// pieces are on their way into shared memory and its cosines and sines, which serve every head, are formed: one barrier a token.
// Into 4 bits, turned keys pass to further warps through shared memory, which round groups of 16 a token behind.
//
// Measured (8 prompts of 1000 to 2000 tokens, 32 heads and 8 key heads of 128): 51 us in 16 bits, 6.1 TB/s of a measured 6.65; a CTA
// that takes one token and loads after its angles 84.  8000 tokens of 20 heads of 192, 64 of them turned: 18.5 us, 6.65 TB/s.  Into 4 bits
// 66 us (111), 5.0 TB/s, 59 where the values held are not wanted: 2.6 of 4 instructions a cycle, of the exact products and the rounding, the
// rest waits at a token's barrier.  Two numbers an instruction (f32x2) took 8 % off it.  Pieces are copied to shared memory rather than loaded ahead into registers: the copies of values from one
// iteration to the next waited for them (4 bits 86).  The table of angles lies in shared memory and a warp finds the places of 32 tokens
// at once, as loads that depend on one another took longer than the rest of an iteration (4 bits 86, 16 bits 56).
#include <algorithm>
#include <cmath>

#include "kv_attention.cuh"
#include "kv_q4.cuh"

namespace pkv {

namespace {

constexpr int kMaxRot = 512;             // rotated elements of a head

// ---------------------------------------------------------------------------
// Cosine and sine of 256 angles a turn in two floats each, from their Taylor series in 64 bits at compile time.
// ---------------------------------------------------------------------------
constexpr double kPi = 3.14159265358979323846;

constexpr double series(double x, bool sine)  // |x| <= pi / 4
{
    double term = sine ? x : 1.0, sum = 0.0;
    for (int n = sine ? 1 : 0; n < 26; n += 2) {
        sum += term;
        term *= -x * x / ((n + 1) * (n + 2));
    }
    return sum;
}

constexpr double turn256(int i, bool sine)
{
    // quarter turns and a remainder of at most an eighth of a turn
    const int q = ((i + 32) >> 6) & 3, r = ((i + 32) & 63) - 32;
    const double x = r * (kPi / 128), c = series(x, false), s = series(x, true);
    const double co = q == 0 ? c : q == 1 ? -s : q == 2 ? -c : s, si = q == 0 ? s : q == 1 ? c : q == 2 ? -s : -c;
    return sine ? si : co;
}

struct Turns {
    float v[256][4];  // cosine, sine, what their rounding leaves
    constexpr Turns() : v()
    {
        for (int i = 0; i < 256; i++) {
            const double c = turn256(i, false), s = turn256(i, true);
            v[i][0] = (float)c;
            v[i][1] = (float)s;
            v[i][2] = (float)(c - (double)(float)c);
            v[i][3] = (float)(s - (double)(float)s);
        }
    }
};

__device__ const __align__(16) Turns g_turns = Turns();

struct Angle {
    float c, s, cl, sl;  // cosine, sine; what their rounding leaves
};

// x + y and what its rounding leaves (Knuth).
__device__ __forceinline__ float sum2(float x, float y, float &left)
{
    const float s = __fadd_rn(x, y), t = __fadd_rn(s, -x);
    left = __fadd_rn(__fadd_rn(x, -__fadd_rn(s, -t)), __fadd_rn(y, -t));
    return s;
}

// m cos, m sin of the sum of an angle of the table and a rest of at most pi / 256, in 2^-64 turns, whose sine and cosine take two
// terms more than themselves.  In one float each, off by little more than their rounding:
__device__ __forceinline__ float2 plain_angle_of(const float4 &t, int64_t rest, float m)
{
    const float x = (float)(int32_t)(rest >> 32) * (float)(2 * kPi / 4294967296.0);
    const float x2 = x * x, s = fmaf(x * x2, -1.0f / 6, x), c = x2 * fmaf(x2, 1.0f / 24, -0.5f);
    return make_float2(m * (t.x + fmaf(t.x, c, fmaf(-t.y, s, t.z))), m * (t.y + fmaf(t.y, c, fmaf(t.x, s, t.w))));
}

// ... and in two:
__device__ __forceinline__ Angle angle_of(const float4 &t, int64_t d, float m)
{
    // the rest in radians: the upper 24 bits of d are exact in 32-bit floating point
    constexpr double kHi = 2 * kPi / 4294967296.0;
    constexpr float k1 = (float)kHi, k1l = (float)(kHi - (double)k1), k2 = (float)(kHi / 4294967296.0);
    const float a = (float)(int32_t)(d >> 32), b = (float)(uint32_t)d;
    float x = __fmul_rn(a, k1), xl = fmaf(a, k1l, fmaf(a, k1, -x));
    xl = fmaf(b, k2, xl);
    const float x0 = x;
    x = __fadd_rn(x0, xl);
    xl = __fadd_rn(xl, -__fadd_rn(x, -x0));
    const float x2 = __fmul_rn(x, x);
    const float sl = fmaf(__fmul_rn(x, x2), fmaf(x2, 1.0f / 120, -1.0f / 6), xl);            // sine: x + sl
    const float ch = -0.5f * x2;                                                             // cosine: 1 + ch + cl
    const float cl = fmaf(__fmul_rn(x2, x2), 1.0f / 24, fmaf(-x, xl, -0.5f * fmaf(x, x, -x2)));
    Angle o;
    // cosine t.x (1 + ch) - t.y x and sine t.y (1 + ch) + t.x x, the large products with what their rounding leaves
    float e, p = __fmul_rn(t.y, x), pe = fmaf(t.y, x, -p), s = sum2(t.x, -p, e);
    float lo = fmaf(t.x, ch, fmaf(t.x, cl, fmaf(-t.y, sl, fmaf(-t.w, x, fmaf(t.z, ch, t.z + (e - pe))))));
    o.c = __fadd_rn(s, lo);
    o.cl = __fadd_rn(lo, -__fadd_rn(o.c, -s));
    p = __fmul_rn(t.x, x), pe = fmaf(t.x, x, -p), s = sum2(t.y, p, e);
    lo = fmaf(t.y, ch, fmaf(t.y, cl, fmaf(t.x, sl, fmaf(t.z, x, fmaf(t.w, ch, t.w + (e + pe))))));
    o.s = __fadd_rn(s, lo);
    o.sl = __fadd_rn(lo, -__fadd_rn(o.s, -s));
    if (m != 1.0f) {
        const float c = __fmul_rn(o.c, m), si = __fmul_rn(o.s, m);
        o.cl = fmaf(o.cl, m, fmaf(o.c, m, -c));
        o.sl = fmaf(o.sl, m, fmaf(o.s, m, -si));
        o.c = c, o.s = si;
    }
    return o;
}

// Two 32-bit numbers that one instruction adds or multiplies, each result rounded by itself.
using Two = uint64_t;

__device__ __forceinline__ Two two(float a, float b)
{
    Two v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
    return v;
}
__device__ __forceinline__ float2 one_by_one(Two v)
{
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
    return f;
}
__device__ __forceinline__ Two add2(Two a, Two b)
{
    Two v;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
    return v;
}
__device__ __forceinline__ Two mul2(Two a, Two b)
{
    Two v;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
    return v;
}
__device__ __forceinline__ Two fma2(Two a, Two b, Two c)
{
    Two v;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(a), "l"(b), "l"(c));
    return v;
}
__device__ __forceinline__ Two neg2(Two a) { return mul2(a, two(-1.0f, -1.0f)); }
__device__ __forceinline__ Two sub2(Two a, Two b) { return fma2(b, two(-1.0f, -1.0f), a); }

// a c + b s of two-float c and s (what their rounding leaves in cl and sl), rounded once.
__device__ __forceinline__ Two turned(Two a, Two b, Two c, Two s, Two cl, Two sl)
{
    const Two p = mul2(a, c), q = mul2(b, s);
    const Two d = add2(p, q), t = sub2(d, p);  // d and what its rounding leaves (Knuth)
    const Two e = add2(sub2(p, sub2(d, t)), sub2(q, t));
    const Two pq = add2(fma2(a, c, neg2(p)), fma2(b, s, neg2(q)));
    return add2(d, add2(e, add2(pq, fma2(a, cl, mul2(b, sl)))));
}

// One set of heads: [tokens, heads, dim] rows with byte strides.
struct Rows {
    const char *in;
    char *out;
    int64_t in_token, in_head, out_token, out_head;
};

// A plane of the cache that takes new rows.
struct Plane {
    char *base;
    int64_t block_stride, token_stride;
    int32_t num_blocks;
};

struct Params {
    Rows q, k, v;  // k.out, v.out: the held values of a 4-bit write, may be null
    Plane kp, vp;
    const int32_t *token_req, *token_pos, *rope_pos;
    const int32_t *table;
    int64_t table_stride;
    const uint64_t *turns;
    int32_t n_reqs, max_blocks;
    int32_t heads, kv_heads, dk, dv;
    int32_t half, offset;  // pairs of a head, its first rotated element
    float magnitude;
    int32_t inverse;
    FastDiv block;
    // what a head consists of: items of 16 elements that rotate (8 pairs), items that do not, groups of 16 for 4 bits
    int32_t n_turn, n_plain, n_v, k_groups, v_groups;
    FastDiv by_turn, by_plain, by_v, by_k_groups, by_v_groups;
    int64_t n_tokens;
    int32_t step;         // tokens that are worked on at a time
    FastDiv chunks;       // CTAs that share a token
    int32_t chunk_heads;  // heads of each, for 4 bits
    int32_t movers;       // threads that rotate and copy; the others round to 4 bits
    int32_t loaders;      // threads that load: all but those that round keys
    float k_scale, v_scale, k_inv, v_inv;
    int *err;
};

template <bool Bf16>
__device__ __forceinline__ float2 unpack2(uint32_t v)
{
    if (Bf16) return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
    float2 f;
    asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}" : "=f"(f.x), "=f"(f.y) : "r"(v));
    return f;
}

// A group of 16 elements to 4 bits: its codes, its scale, and (held) the values they stand for.
template <bool Bf16>
__device__ __forceinline__ void quantise(const uint4 (&in)[2], float inv, float scale, char *codes, char *unit, char *held)
{
    const uint32_t w[8] = {in[0].x, in[0].y, in[0].z, in[0].w, in[1].x, in[1].y, in[1].z, in[1].w};
    Two y[8];  // the negatives of what is rounded
    float most = 0.0f;
    const Two by = two(-inv, -inv);
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const float2 f = unpack2<Bf16>(w[i]);
        y[i] = mul2(two(f.x, f.y), by);
        const float2 g = one_by_one(y[i]);
        most = fmaxf(most, fmaxf(fabsf(g.x), fabsf(g.y)));
    }
    const uint32_t b = q4_scale_of(most);
    const uint32_t ss = e4m3x2_to_f16(b * 0x101u);
    const float s = unpack2<false>(ss).x;
    if (most > 6.0f * s * 2) {  // far outside: the largest code, also for infinities
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const float2 f = one_by_one(y[i]);
            y[i] = two(fminf(fmaxf(f.x, -12.0f * s), 12.0f * s), fminf(fmaxf(f.y, -12.0f * s), 12.0f * s));
        }
    }
    // y / s: a quotient that is exact where it can be decides the ties.  One step on the product with the reciprocal gives the
    // rounded quotient (Markstein 1990); with these signs it keeps that of a zero.
    const float r = -__frcp_rn(s);
    const Two rr = two(r, r), s2 = two(s, s);
    uint32_t c[2];
#pragma unroll
    for (int h = 0; h < 2; h++) {
        float z[8];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const Two z0 = mul2(y[4 * h + i], rr);
            const float2 f = one_by_one(fma2(fma2(z0, s2, y[4 * h + i]), rr, z0));
            z[2 * i] = f.x, z[2 * i + 1] = f.y;
        }
        c[h] = f32_to_q4(z);
    }
    if (codes != nullptr) {
        *reinterpret_cast<uint2 *>(codes) = make_uint2(c[0], c[1]);
        *unit = (char)b;
    }
    if (held != nullptr) {
#pragma unroll
        for (int h = 0; h < 2; h++) {
            uint32_t v[4], o[4];
            q4_to_f16(c[h], v);
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const float2 f = unpack2<false>(mul_f16x2(v[i], ss));
                o[i] = pack2<Bf16>(__fmul_rn(f.x, scale), __fmul_rn(f.y, scale));
            }
            reinterpret_cast<uint4 *>(held)[h] = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
}

constexpr int kAngles = kMaxRot / 2;
constexpr int kSmBytes = 228 * 1024;  // of an SM's shared memory

// 16 bytes into shared memory, by themselves.
__device__ __forceinline__ void copy_async(uint32_t to, const char *from)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}

// Threads of a CTA at most and CTAs on an SM, which give the registers of a thread.  16 bits: 64 registers; the prompts above with 256 x 4
// 51.0 us, 128 x 8 52.5, 192 x 5 50.9 (but 18.5, 19.0, 19.8 for 8000 tokens without a cache), 128 x 9 with 56 registers 54.5.  4 bits: a
// token's keys and their groups best lie in one CTA; 72 registers with 448 x 2 65 us, 64 with 512 x 2 82 (they do not fit).
template <bool Q4>
struct Shape {
    static constexpr int kThreads = Q4 ? 448 : 256, kCtas = Q4 ? 2 : 4;
};

template <bool Q4>
struct Angles {
    float v[Q4 ? 4 : 2][kAngles];  // cosines, sines, what their rounding leaves
};

template <bool Bf16, bool Interleaved, bool Q4>
__global__ void __launch_bounds__(Shape<Q4>::kThreads, Shape<Q4>::kCtas) rotate_kernel(const __grid_constant__ Params p)
{
    __shared__ __align__(16) Angles<Q4> angles[2];
    __shared__ __align__(16) float4 near_angles[256];
    // by a token's number here, modulo 64: its rows of keys and values (null: it has none), its position
    __shared__ char *rows[64][2];
    __shared__ int32_t positions[64];
    extern __shared__ __align__(16) char stage[];  // every thread's pieces, then the turned keys
    const int tid = threadIdx.x, threads = blockDim.x;
    const uint32_t first = fdiv(blockIdx.x, p.chunks), chunk = blockIdx.x - first * p.chunks.d;
    const int count = (int)(((uint32_t)p.n_tokens - first - 1) / (uint32_t)p.step) + 1;  // of tokens that this CTA works on
    const int loaders = Q4 ? p.loaders : threads;
    char *const keys = stage + 64 * loaders;
    // The thread's item: two pieces of 16 bytes of a head, `d1` bytes apart, that move together (apart, so that a warp's are in runs).
    const bool mover = !Q4 || tid < p.movers;
    const int h0 = Q4 ? (int)chunk * p.chunk_heads : 0, n_heads = Q4 ? min(p.chunk_heads, p.heads + p.kv_heads - h0) : p.heads + p.kv_heads;
    const int n_keys = Q4 ? max(min(p.kv_heads - h0, n_heads), 0) : 0;  // key heads of this CTA
    enum { kNone, kOut, kKeyRow, kValueRow, kKeys, kKeyGroup, kValueGroup } what = kNone;
    bool turn = false, two_pieces = true;
    const char *src = nullptr;
    int64_t in_step = 0, at_out = 0, out_step = 0;  // at_out: from the row, from `keys`, or an address
    int d1 = 16, n = 0, dim = p.dk;
    if (mover) {
        int i = Q4 ? tid : (int)(chunk * threads) + tid, h = 0, o0 = 0;
        const int turns = n_heads * p.n_turn, plains = n_heads * p.n_plain;
        if (i < turns) {
            h = (int)fdiv((uint32_t)i, p.by_turn), n = i - h * p.n_turn;
            turn = true;
            o0 = p.offset + n * 8;
            d1 = Interleaved ? p.n_turn * 16 : p.half * 2;
            two_pieces = !Interleaved || (n + p.n_turn) * 4 < p.half;
            what = kOut;
        } else if ((i -= turns) < plains) {
            h = (int)fdiv((uint32_t)i, p.by_plain);
            o0 = (i - h * p.n_plain) * 8;
            int o1 = o0 + p.n_plain * 8;
            two_pieces = o1 < p.dk - 2 * p.half;
            if (o0 >= p.offset) o0 += 2 * p.half;
            if (o1 >= p.offset) o1 += 2 * p.half;
            d1 = (o1 - o0) * 2;
            what = kOut;
        } else if (!Q4 && (i -= plains) < p.kv_heads * p.n_v) {
            h = (int)fdiv((uint32_t)i, p.by_v);
            o0 = (i - h * p.n_v) * 8;
            d1 = p.n_v * 16;
            two_pieces = o0 + p.n_v * 8 < p.dv;
            src = p.v.in + h * p.v.in_head, in_step = p.v.in_token;
            at_out = ((int64_t)h * p.dv + o0) * 2;
            what = kValueRow;
        }
        if (what == kOut) {  // keys come before queries
            const int g = h0 + h - p.kv_heads;
            if (g < 0) {
                src = p.k.in + (h0 + h) * p.k.in_head, in_step = p.k.in_token;
                at_out = ((int64_t)h * p.dk + o0) * 2;
                what = Q4 ? kKeys : kKeyRow;
            } else {
                src = p.q.in + g * p.q.in_head, in_step = p.q.in_token;
                at_out = (int64_t)(p.q.out + g * p.q.out_head + o0 * 2), out_step = p.q.out_token;
                if (!turn && p.q.out == p.q.in && out_step == in_step && p.q.out_head == p.q.in_head) what = kNone;  // in place
            }
        }
        src += o0 * 2;
    } else {
        const int ks = n_keys * p.k_groups;
        int i = tid - p.movers;
        if (i < ks) {
            at_out = h0 * p.k_groups + i;
            n = i;
            out_step = p.k.out_token, what = kKeyGroup;
        } else if ((i -= ks) < n_keys * p.v_groups) {
            const int h = (int)fdiv((uint32_t)i, p.by_v_groups);
            src = p.v.in + (h0 + h) * p.v.in_head + (i - h * p.v_groups) * 32, in_step = p.v.in_token;
            at_out = h0 * p.v_groups + i;
            dim = p.dv, out_step = p.v.out_token, what = kValueGroup;
        }
    }
    const bool loads = what != kNone && what != kKeyGroup, group = what >= kKeyGroup;
    // The thread's own pairs: the first with its frequency at hand.  (4 bits: the threads that turn queries come first, as keys take longer.)
    const int own = !mover ? p.half : !Q4 ? tid : tid - n_keys * p.n_turn + (tid < n_keys * p.n_turn ? p.movers : 0);
    const int owners = Q4 ? p.movers : threads;
    const auto angle = [](int32_t pos, uint64_t turn) { return (uint64_t)(int64_t)pos * turn + (1ull << 55); };  // rounded to the table's by its upper byte
    const auto put_angle = [&](Angles<Q4> &to, int i, uint64_t u, const float4 &close) {
        const int64_t rest = (int64_t)(u & ((1ull << 56) - 1)) - (1ll << 55);
        // four pairs side by side; halves: a piece's first four pairs before all pieces' second four, so that a warp reads runs
        const int at = Interleaved ? i : (((i >> 2 & 1) * p.n_turn + (i >> 3)) << 2) + (i & 3);
        if constexpr (Q4) {
            const Angle a = angle_of(close, rest, p.magnitude);
            to.v[0][at] = a.c, to.v[1][at] = a.s, to.v[2][at] = a.cl, to.v[3][at] = a.sl;
        } else {
            const float2 a = plain_angle_of(close, rest, p.magnitude);
            to.v[0][at] = a.x, to.v[1][at] = p.inverse ? -a.y : a.y;
        }
    };
    // the places of 32 tokens from number `at` on, by one warp: a wait for three loads in a row, one in 32 tokens
    const auto place_tokens = [&](int at) {
        at += tid & 31;
        if (at >= count) return;
        const int64_t t = first + (int64_t)at * p.step;
        int32_t req = -1, pos = -1;
        if (p.kv_heads) req = __ldg(p.token_req + t), pos = __ldg(p.token_pos + t);
        positions[at & 63] = __ldg(p.rope_pos + t);
        if (p.kv_heads == 0) return;
        int page = -1, slot = 0;
        if (req >= 0 && req < p.n_reqs && pos >= 0) {
            const uint32_t col = fdiv((uint32_t)pos, p.block);
            if (col < (uint32_t)p.max_blocks) {
                page = __ldg(p.table + (int64_t)req * p.table_stride + col);
                slot = (int)((uint32_t)pos - col * p.block.d);
            }
        }
        if (page < 0)
            set_error(p.err, KV_DERR_TABLE);
        else if (page >= p.kp.num_blocks || (p.dv && page >= p.vp.num_blocks))
            set_error(p.err, KV_DERR_SLOT), page = -1;
        rows[at & 63][0] = page < 0 ? nullptr : p.kp.base + (int64_t)page * p.kp.block_stride + (int64_t)slot * p.kp.token_stride;
        rows[at & 63][1] = page < 0 ? nullptr : p.vp.base + (int64_t)page * p.vp.block_stride + (int64_t)slot * p.vp.token_stride;
    };
    grid_dep_entry();
    const uint64_t own_turn = own < p.half ? __ldg(p.turns + own) : 0;
    src += first * in_step;
    const char *src1 = src + d1;
    if (what == kOut) at_out += first * out_step;
    int64_t done = first * out_step;
    out_step *= p.step;
    in_step *= p.step;
    const int mine = mover ? tid : what == kValueGroup ? tid - n_keys * p.k_groups : 0;  // the thread's place among those that load
    const auto load = [&](int to) {
        if (loads) {
            const uint32_t at = smem_addr(stage) + ((to & 1) * 2 * loaders + mine) * 16;
            copy_async(at, src);
            if (two_pieces) copy_async(at + loaders * 16, src1);
            src += in_step, src1 += in_step;
        }
    };
    if (mover) load(0);
    if (count > 1)
        for (int i = tid; i < 256; i += threads) copy_async(smem_addr(near_angles + i), reinterpret_cast<const char *>(g_turns.v[i]));
    if (tid >= threads - 32) place_tokens(0);
    for (int i = own; i < p.half; i += owners) {
        const uint64_t u = angle(__ldg(p.rope_pos + first), i == own ? own_turn : __ldg(p.turns + i));
        put_angle(angles[0], i, u, __ldg(reinterpret_cast<const float4 *>(g_turns.v[u >> 56])));
    }
    asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
    __syncthreads();
    for (int it = 0; it < count + Q4; it++) {
        // the next token's loads are under way while this one's heads are turned (values are rounded a token behind)
        const bool more = it + 1 < count;
        if (mover ? more : it < count) load(mover ? it + 1 : it);
        asm volatile("cp.async.commit_group;" ::: "memory");
        if ((it & 31) == 16 && tid >= threads - 32) place_tokens(it + 16);
        if (more)
            for (int i = own; i < p.half; i += owners) {
                const uint64_t u = angle(positions[(it + 1) & 63], i == own ? own_turn : __ldg(p.turns + i));
                put_angle(angles[(it + 1) & 1], i, u, near_angles[u >> 56]);
            }
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        const int slot = (mover ? it : it - 1) & 1;
        uint4 x = *reinterpret_cast<const uint4 *>(stage + (slot * 2 * loaders + mine) * 16);
        uint4 y = *reinterpret_cast<const uint4 *>(stage + ((slot * 2 + 1) * loaders + mine) * 16);
        if (!group && what != kNone && (!Q4 || it < count)) {
            char *to = reinterpret_cast<char *>(at_out);
            if (what == kOut) {
                at_out += out_step;
            } else if (what == kKeys) {
                to = keys + (it & 1) * (n_keys * p.dk * 2) + at_out;
            } else {
                char *const row = rows[it & 63][what == kValueRow];
                to = row == nullptr ? nullptr : row + at_out;
            }
            if (turn) {
                const Angles<Q4> &g = angles[it & 1];
                const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
                uint32_t ox[4], oy[4];
#pragma unroll
                for (int j = 0; j < 2; j++) {
                    const int ga = (j * p.n_turn + n) * 4;
                    const ulonglong2 c = *reinterpret_cast<const ulonglong2 *>(&g.v[0][ga]), s = *reinterpret_cast<const ulonglong2 *>(&g.v[1][ga]);
                    ulonglong2 cl = {}, sl = {};
                    const bool exact = Q4 && what == kKeys;
                    if constexpr (Q4)
                        if (exact) cl = *reinterpret_cast<const ulonglong2 *>(&g.v[2][ga]), sl = *reinterpret_cast<const ulonglong2 *>(&g.v[3][ga]);
#pragma unroll
                    for (int k = 0; k < 2; k++) {
                        // two pairs (a, b)
                        Two a, b, na, nb;
                        const uint32_t w0 = Interleaved ? (j ? ys : xs)[2 * k] : xs[2 * j + k], w1 = Interleaved ? (j ? ys : xs)[2 * k + 1] : ys[2 * j + k];
                        const float2 u = unpack2<Bf16>(w0), v = unpack2<Bf16>(w1);
                        a = Interleaved ? two(u.x, v.x) : two(u.x, u.y);
                        b = Interleaved ? two(u.y, v.y) : two(v.x, v.y);
                        const Two cc = k ? c.y : c.x, sn = k ? s.y : s.x;
                        if (exact) {
                            const Two ccl = k ? cl.y : cl.x, snl = k ? sl.y : sl.x;
                            na = turned(a, neg2(b), cc, sn, ccl, snl);
                            nb = turned(a, b, sn, cc, snl, ccl);
                        } else {
                            na = fma2(b, neg2(sn), mul2(a, cc));
                            nb = fma2(a, sn, mul2(b, cc));
                        }
                        const float2 fa = one_by_one(na), fb = one_by_one(nb);
                        if (Interleaved) {
                            (j ? oy : ox)[2 * k] = pack2<Bf16>(fa.x, fb.x);
                            (j ? oy : ox)[2 * k + 1] = pack2<Bf16>(fa.y, fb.y);
                        } else {
                            ox[2 * j + k] = pack2<Bf16>(fa.x, fa.y);
                            oy[2 * j + k] = pack2<Bf16>(fb.x, fb.y);
                        }
                    }
                }
                x = make_uint4(ox[0], ox[1], ox[2], ox[3]);
                y = make_uint4(oy[0], oy[1], oy[2], oy[3]);
            }
            if (to != nullptr) {
                *reinterpret_cast<uint4 *>(to) = x;
                if (two_pieces) *reinterpret_cast<uint4 *>(to + d1) = y;
            }
        }
        if constexpr (Q4) {
            if (group && it > 0) {  // a token behind: its keys are in shared memory
                const bool key = what == kKeyGroup;
                uint4 in[2] = {x, y};
                if (key) {
                    const uint4 *from = reinterpret_cast<const uint4 *>(keys + ((it - 1) & 1) * (n_keys * p.dk * 2) + n * 32);
                    in[0] = from[0], in[1] = from[1];
                }
                char *const row = rows[(it - 1) & 63][!key], *const held = key ? p.k.out : p.v.out;
                quantise<Bf16>(in, key ? p.k_inv : p.v_inv, key ? p.k_scale : p.v_scale, row ? row + at_out * 8 : nullptr,
                               row ? row + p.kv_heads * dim / 2 + at_out : nullptr, held ? held + done + at_out * 32 : nullptr);
                done += out_step;
            }
        }
        if (it + 1 < count + Q4) __syncthreads();
    }
}

template <bool Bf16, bool Interleaved, bool Q4>
int run_rotate(Params *p, cudaStream_t s)
{
    const DeviceInfo *dev = current_device();
    if (dev == nullptr) return KV_ERR_CUDA;
    const auto warps = [](int64_t n) { return (n + 31) / 32 * 32; };
    const int all = p->heads + p->kv_heads;
    int64_t chunks = 1, threads;
    size_t keys = 0;
    if (Q4) {
        const int each = p->n_turn + p->n_plain, groups = p->k_groups + p->v_groups;
        for (;; chunks++) {
            p->chunk_heads = (int)((all + chunks - 1) / chunks);
            p->movers = (int)warps((int64_t)p->chunk_heads * each);
            threads = p->movers + warps((int64_t)std::min(p->chunk_heads, p->kv_heads) * groups);
            if (threads <= Shape<Q4>::kThreads) break;
        }
        chunks = (all + p->chunk_heads - 1) / p->chunk_heads;
        p->loaders = p->movers + std::min(p->chunk_heads, p->kv_heads) * p->v_groups;
        keys = (size_t)std::min(p->chunk_heads, p->kv_heads) * p->dk * 4;
    } else {
        const int64_t items = (int64_t)all * (p->n_turn + p->n_plain) + (int64_t)p->kv_heads * p->n_v;
        chunks = (items + Shape<Q4>::kThreads - 1) / Shape<Q4>::kThreads;
        threads = warps((items + chunks - 1) / chunks);
    }
    const auto by = [](int n) { return make_fastdiv((uint32_t)std::max(n, 1)); };
    p->by_turn = by(p->n_turn), p->by_plain = by(p->n_plain), p->by_v = by(p->n_v), p->by_k_groups = by(p->k_groups), p->by_v_groups = by(p->v_groups);
    p->chunks = by((int)chunks);
    const size_t smem = keys + 64 * (Q4 ? p->loaders : threads), fixed = 2 * sizeof(Angles<Q4>) + 256 * 16 + 64 * 20 + 1024;
    const int64_t on_sm = std::min<int64_t>(Shape<Q4>::kThreads * Shape<Q4>::kCtas / threads, kSmBytes / (smem + fixed));
    const int64_t at_once = std::max<int64_t>(dev->num_sms * on_sm / chunks, 1);
    p->step = (int)std::min(p->n_tokens, at_once);
    return cuda_status(launch(rotate_kernel<Bf16, Interleaved, Q4>, dim3((unsigned)(p->step * chunks)), dim3((unsigned)threads), smem, s, *p));
}

template <bool Bf16, bool Interleaved>
int pick_rotate(bool q4, Params *p, cudaStream_t s)
{
    return q4 ? run_rotate<Bf16, Interleaved, true>(p, s) : run_rotate<Bf16, Interleaved, false>(p, s);
}

int launch_rotate(int dtype, bool interleaved, bool q4, Params *p, cudaStream_t s)
{
    if (dtype == KV_BF16) return interleaved ? pick_rotate<true, true>(q4, p, s) : pick_rotate<true, false>(q4, p, s);
    return interleaved ? pick_rotate<false, true>(q4, p, s) : pick_rotate<false, false>(q4, p, s);
}

// The rotation's part of the parameters, for heads of `dim` elements.
int fill_rope(Params *p, const kv_rope *r, int dim)
{
    p->magnitude = 1.0f;
    p->n_plain = (dim + 15) / 16;
    if (r == nullptr || r->rot_dim == 0) return KV_OK;
    if (r->rot_dim < 0 || r->rot_offset < 0 || r->turns == nullptr || !std::isfinite(r->magnitude)) return KV_ERR_INVALID_ARG;
    if (r->rot_dim > dim || r->rot_offset > dim - r->rot_dim) return KV_ERR_RANGE;
    if (r->rot_dim % (r->interleaved ? 8 : 16) || r->rot_offset % 8 || ((uintptr_t)r->turns & 7u)) return KV_ERR_ALIGN;
    if (r->rot_dim > kMaxRot) return KV_ERR_UNSUPPORTED;
    p->turns = r->turns;
    p->half = r->rot_dim / 2;
    p->offset = r->rot_offset;
    p->magnitude = r->magnitude;
    p->n_turn = (r->rot_dim + 15) / 16;
    p->n_plain = (dim - r->rot_dim + 15) / 16;
    return KV_OK;
}

int check_heads(int dtype, int heads, int dim)
{
    if (dtype != KV_BF16 && dtype != KV_F16) return KV_ERR_INVALID_ARG;
    if (heads < 0 || dim <= 0) return KV_ERR_INVALID_ARG;
    if (dim % 8) return KV_ERR_ALIGN;
    if (dim > (1 << 16) || heads > (1 << 14)) return KV_ERR_UNSUPPORTED;
    return KV_OK;
}

// What both writes check and fill in.
int fill_write(Params *p, const kv_new_tokens *t, const kv_rope *rope, const kv_cache_desc *k, int k_tensor, int k_plane,
               const kv_cache_desc *v, int v_tensor, int v_plane, bool q4)
{
    if (t == nullptr || t->n_tokens < 0 || t->n_reqs < 0 || t->max_blocks_per_req < 0 || t->bt_row_stride < 0 || t->n_kv_heads <= 0 ||
        t->head_dim_v < 0)
        return KV_ERR_INVALID_ARG;
    int st;
    if ((st = check_heads(t->dtype, t->n_heads, t->head_dim)) != KV_OK) return st;
    if ((st = check_heads(t->dtype, t->n_kv_heads, t->head_dim_v ? t->head_dim_v : 8)) != KV_OK) return st;
    if (t->n_reqs > 1 && t->bt_row_stride < t->max_blocks_per_req) return KV_ERR_INVALID_ARG;
    if ((st = fill_rope(p, rope, t->head_dim)) != KV_OK) return st;
    const auto check = q4 ? check_q4_plane : check_plane;
    if ((st = check(k, k_tensor, k_plane, t->n_kv_heads, t->head_dim)) != KV_OK) return st;
    if (t->head_dim_v) {
        if ((st = check(v, v_tensor, v_plane, t->n_kv_heads, t->head_dim_v)) != KV_OK) return st;
        if (k->block_size != v->block_size) return KV_ERR_INVALID_ARG;
    }
    if (t->n_tokens == 0) return KV_OK;
    if (t->n_tokens >= (1ll << 31)) return KV_ERR_UNSUPPORTED;
    if (t->token_req == nullptr || t->token_pos == nullptr || (t->block_table == nullptr && t->n_reqs > 0 && t->max_blocks_per_req > 0))
        return KV_ERR_INVALID_ARG;
    const DeviceInfo *dev = current_device();
    if (t->n_heads) {
        if ((st = check_rows(t->q, t->q_token_stride, t->q_head_stride)) != KV_OK) return st;
        if ((st = check_rows(t->q_out, t->q_out_token_stride, t->q_out_head_stride)) != KV_OK) return st;
        p->q = Rows{(const char *)t->q, (char *)t->q_out, t->q_token_stride, t->q_head_stride, t->q_out_token_stride, t->q_out_head_stride};
    }
    if ((st = check_rows(t->k, t->k_token_stride, t->k_head_stride)) != KV_OK) return st;
    p->k = Rows{(const char *)t->k, nullptr, t->k_token_stride, t->k_head_stride, 0, 0};
    p->kp = Plane{(char *)k->base[k_tensor] + (k_plane ? k->plane_stride : 0), k->block_stride, k->token_stride, (int32_t)k->num_blocks};
    if (t->head_dim_v) {
        if ((st = check_rows(t->v, t->v_token_stride, t->v_head_stride)) != KV_OK) return st;
        p->v = Rows{(const char *)t->v, nullptr, t->v_token_stride, t->v_head_stride, 0, 0};
        p->vp = Plane{(char *)v->base[v_tensor] + (v_plane ? v->plane_stride : 0), v->block_stride, v->token_stride, (int32_t)v->num_blocks};
        p->n_v = (t->head_dim_v + 15) / 16;
        p->v_groups = t->head_dim_v / 16;
    }
    p->k_groups = t->head_dim / 16;
    p->n_tokens = t->n_tokens;
    p->token_req = t->token_req;
    p->token_pos = t->token_pos;
    p->rope_pos = t->rope_pos ? t->rope_pos : t->token_pos;
    p->table = t->block_table;
    p->table_stride = t->bt_row_stride;
    p->n_reqs = t->n_reqs;
    p->max_blocks = t->max_blocks_per_req;
    p->heads = t->n_heads;
    p->kv_heads = t->n_kv_heads;
    p->dk = t->head_dim;
    p->dv = t->head_dim_v;
    p->block = make_fastdiv((uint32_t)k->block_size);
    if (dev == nullptr) return KV_ERR_CUDA;
    p->err = dev->err_word;
    return KV_OK;
}

}  // namespace

int check_q4_plane(const kv_cache_desc *c, int tensor, int plane, int heads, int dim)
{
    const int st = check_cache(c);
    if (st != KV_OK) return st;
    if (tensor < 0 || tensor >= c->n_tensors || plane < 0 || plane >= c->n_planes) return KV_ERR_INVALID_ARG;
    if (dim % 32) return KV_ERR_ALIGN;
    if (dim > kQ4MaxDim) return KV_ERR_UNSUPPORTED;
    if (q4_row_bytes(heads, dim) != c->row_bytes || c->num_blocks == 0) return KV_ERR_INVALID_ARG;
    if (c->num_blocks >= (1ll << 31) || c->token_stride >= (1ll << 40) || c->block_stride >= (1ll << 40)) return KV_ERR_UNSUPPORTED;
    return KV_OK;
}

int preload_rotate_kernels()
{
    return load_kernels(rotate_kernel<false, false, false>, rotate_kernel<false, false, true>, rotate_kernel<false, true, false>,
                        rotate_kernel<false, true, true>, rotate_kernel<true, false, false>, rotate_kernel<true, false, true>,
                        rotate_kernel<true, true, false>, rotate_kernel<true, true, true>);
}

}  // namespace pkv

using namespace pkv;

extern "C" {

int kv_rope_frequencies(int32_t rot_dim, double base, const kv_rope_scaling *scaling, uint64_t *turns_out, float *magnitude_out)
{
    const int kind = scaling ? scaling->kind : KV_ROPE_PLAIN;
    if (turns_out == nullptr || rot_dim <= 0 || rot_dim % 2 || !(base > 1.0) || !std::isfinite(base) || kind < KV_ROPE_PLAIN || kind > KV_ROPE_YARN)
        return KV_ERR_INVALID_ARG;
    const double f = kind == KV_ROPE_PLAIN ? 1.0 : scaling->factor, length = scaling ? scaling->original_length : 0.0;
    if (!(f > 0.0) || !std::isfinite(f)) return KV_ERR_INVALID_ARG;
    const bool banded = kind == KV_ROPE_BANDS || kind == KV_ROPE_YARN;
    if (banded && (!(length > 0.0) || !std::isfinite(length) || !(scaling->slow > 0.0) || !(scaling->fast > scaling->slow) || !std::isfinite(scaling->fast)))
        return KV_ERR_INVALID_ARG;
    constexpr double kTurn = 6.283185307179586476925;
    const double d = rot_dim;
    if (kind == KV_ROPE_BASE) {
        if (rot_dim <= 2) return KV_ERR_INVALID_ARG;
        base *= std::pow(f, d / (d - 2.0));
    }
    double low = 0.0, high = 0.0;
    if (kind == KV_ROPE_YARN) {  // pairs that turn `fast` and `slow` times over the original length
        low = std::fmax(std::floor(d * std::log(length / (scaling->fast * kTurn)) / (2.0 * std::log(base))), 0.0);
        high = std::fmin(std::ceil(d * std::log(length / (scaling->slow * kTurn)) / (2.0 * std::log(base))), d - 1.0);
    }
    const auto frequency = [&](int i) {
        double w = std::pow(base, -2.0 * i / d), mix = 1.0;  // mix: how much of the frequency stays as it is
        if (kind == KV_ROPE_LINEAR) mix = 0.0;
        if (kind == KV_ROPE_BANDS) mix = (length * w / kTurn - scaling->slow) / (scaling->fast - scaling->slow);
        if (kind == KV_ROPE_YARN) mix = 1.0 - (i - low) / std::fmax(high - low, 1e-3);
        mix = std::fmin(std::fmax(mix, 0.0), 1.0);
        return kind == KV_ROPE_BASE ? w : w * mix + w / f * (1.0 - mix);
    };
    for (int i = 0; i < rot_dim / 2; i++)  // a factor near 0 takes them out of 64 bits
        if (!std::isfinite(frequency(i))) return KV_ERR_INVALID_ARG;
    for (int i = 0; i < rot_dim / 2; i++) {
        // of a turn, whole ones dropped
        const double t = std::nearbyint(std::ldexp(std::fmod(frequency(i) / kTurn, 1.0), 64));
        turns_out[i] = t >= 18446744073709551616.0 ? 0 : (uint64_t)t;
    }
    if (magnitude_out) *magnitude_out = (float)(kind == KV_ROPE_YARN && f > 1.0 ? 0.1 * std::log(f) + 1.0 : 1.0);
    return KV_OK;
}

int kv_rotate(int32_t dtype, int32_t n_heads, int32_t head_dim, const void *x, int64_t token_stride, int64_t head_stride, void *out,
              int64_t out_token_stride, int64_t out_head_stride, int64_t n_tokens, const int32_t *token_pos, const kv_rope *rope, int32_t inverse,
              kv_stream_t stream)
{
    Params p = {};
    int st = check_heads(dtype, n_heads, head_dim);
    if (st != KV_OK) return st;
    if (n_tokens < 0 || rope == nullptr) return KV_ERR_INVALID_ARG;
    if ((st = fill_rope(&p, rope, head_dim)) != KV_OK) return st;
    if (n_tokens >= (1ll << 31)) return KV_ERR_UNSUPPORTED;
    if (n_tokens == 0 || n_heads == 0) return KV_OK;
    if (token_pos == nullptr) return KV_ERR_INVALID_ARG;
    if ((st = check_rows(x, token_stride, head_stride)) != KV_OK) return st;
    if ((st = check_rows(out, out_token_stride, out_head_stride)) != KV_OK) return st;
    p.q = Rows{(const char *)x, (char *)out, token_stride, head_stride, out_token_stride, out_head_stride};
    p.rope_pos = token_pos;
    p.heads = n_heads;
    p.dk = head_dim;
    p.inverse = inverse != 0;
    p.n_tokens = n_tokens;
    return launch_rotate(dtype, rope->interleaved != 0, false, &p, (cudaStream_t)stream);
}

int kv_q4_row_bytes(int32_t heads, int32_t head_dim, int32_t *bytes_out)
{
    if (bytes_out == nullptr || heads <= 0 || head_dim <= 0) return KV_ERR_INVALID_ARG;
    if (head_dim % 32) return KV_ERR_ALIGN;
    if (head_dim > kQ4MaxDim || heads > (1 << 14)) return KV_ERR_UNSUPPORTED;
    *bytes_out = (int32_t)q4_row_bytes(heads, head_dim);
    return KV_OK;
}

int kv_rotate_write(const kv_new_tokens *tokens, const kv_rope *rope, const kv_cache_desc *k, int32_t k_tensor, int32_t k_plane,
                    const kv_cache_desc *v, int32_t v_tensor, int32_t v_plane, kv_stream_t stream)
{
    Params p = {};
    const int st = fill_write(&p, tokens, rope, k, k_tensor, k_plane, v, v_tensor, v_plane, false);
    if (st != KV_OK || tokens->n_tokens == 0) return st;
    return launch_rotate(tokens->dtype, rope && rope->interleaved, false, &p, (cudaStream_t)stream);
}

int kv_rotate_write_q4(const kv_new_tokens *tokens, const kv_rope *rope, const kv_cache_desc *k, int32_t k_tensor, int32_t k_plane,
                       const kv_cache_desc *v, int32_t v_tensor, int32_t v_plane, float k_scale, float v_scale, void *k_held, void *v_held,
                       kv_stream_t stream)
{
    Params p = {};
    if (tokens != nullptr && tokens->head_dim_v == 0) return KV_ERR_UNSUPPORTED;
    if (!good_scale(k_scale) || !good_scale(v_scale)) return KV_ERR_INVALID_ARG;
    if (!aligned16(k_held) || !aligned16(v_held)) return KV_ERR_ALIGN;
    const int st = fill_write(&p, tokens, rope, k, k_tensor, k_plane, v, v_tensor, v_plane, true);
    if (st != KV_OK || tokens->n_tokens == 0) return st;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.k_inv = (float)(1.0 / k_scale);
    p.v_inv = (float)(1.0 / v_scale);
    p.k.out = (char *)k_held;
    p.v.out = (char *)v_held;
    p.k.out_token = (int64_t)tokens->n_kv_heads * tokens->head_dim * 2;
    p.v.out_token = (int64_t)tokens->n_kv_heads * tokens->head_dim_v * 2;
    return launch_rotate(tokens->dtype, rope && rope->interleaved, true, &p, (cudaStream_t)stream);
}

}  // extern "C"
