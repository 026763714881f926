// How the attention kernels cut a ragged batch into work, on the device, from the lengths alone.
//
// A request's query rows are its (token, head of the group) pairs, token-major: row = token * group +
// head.  Rows are cut into units of `unit_rows`; a unit of one key head needs the key tiles of
// `tile` keys between the first key that its first token sees and the last that its last token sees.
// Laid end to end (request, key head, unit), all units' tiles form one line; CTA c of `parts` takes
// the c-th equal piece of it.  A piece may begin and end inside a unit: those two fragments go to the
// workspace, and whichever CTA finishes the unit's last one joins them.  So the split follows the lengths, not the launch: one
// grid serves a captured graph whatever the lengths become, and long contexts and few rows fill the
// GPU as well as many short requests do.
#pragma once

#include <cstdint>

#include "kv_common.cuh"

namespace pkv {

struct Batch {
    const int32_t *q_offsets;  // [n_reqs + 1]
    const int32_t *kv_lens;    // [n_reqs]
    int32_t n_reqs;
    int32_t n_tokens;    // capacity: q_offsets entries are clamped to it
    int32_t max_tokens;  // capacity of a table row in tokens: kv_lens entries are clamped to it
    int32_t kv_heads;
    int32_t unit_rows;
    int32_t tile;  // keys of one tile
    int32_t causal;
    int32_t window;  // 0: none
    FastDiv group;   // query heads of a key head
    int *err;
};

struct Request {
    int32_t q0, q_len, len;
    int32_t rows, units;
};

struct Unit {
    int32_t row0, rows;  // rows of the request
    int32_t lo, hi;      // keys that some row sees
    int32_t tile0, tiles;  // key tiles (absolute index of the first, count)
};

__device__ __forceinline__ Request load_request(const Batch &b, int r, bool report = false)
{
    Request q;
    const int a = __ldg(b.q_offsets + r), e = __ldg(b.q_offsets + r + 1), n = __ldg(b.kv_lens + r);
    q.q0 = min(max(a, 0), b.n_tokens);
    const int end = min(max(e, q.q0), b.n_tokens);
    q.q_len = end - q.q0;
    q.len = min(max(n, 0), b.max_tokens);
    q.rows = q.q_len * (int)b.group.d;
    q.units = (q.rows + b.unit_rows - 1) / b.unit_rows;
    if (report && (a != q.q0 || e != end || (r == 0 && a != 0))) set_error(b.err, KV_DERR_LIST);
    if (report && n != q.len) set_error(b.err, KV_DERR_TABLE);
    return q;
}

// Keys [lo, hi) that query token t of the request sees.
__device__ __forceinline__ void sees(const Batch &b, const Request &q, int t, int &lo, int &hi)
{
    const int pos = q.len - q.q_len + t;
    hi = b.causal ? min(q.len, pos + 1) : q.len;
    hi = max(hi, 0);
    lo = b.window ? min(max(pos - b.window + 1, 0), hi) : 0;
}

__device__ __forceinline__ Unit make_unit(const Batch &b, const Request &q, int j)
{
    Unit u;
    u.row0 = j * b.unit_rows;
    u.rows = min(b.unit_rows, q.rows - u.row0);
    int x;
    sees(b, q, (int)fdiv((uint32_t)u.row0, b.group), u.lo, x);
    sees(b, q, (int)fdiv((uint32_t)(u.row0 + u.rows - 1), b.group), x, u.hi);
    u.tile0 = u.lo / b.tile;
    u.tiles = u.hi > u.lo ? (u.hi + b.tile - 1) / b.tile - u.tile0 : 0;
    return u;
}

// A unit that sees nothing still takes one step of the line: its rows have to be written.
__device__ __forceinline__ int unit_cost(const Unit &u) { return max(1, u.tiles); }

__device__ __forceinline__ long long head_cost(const Batch &b, const Request &q)
{
    long long n = 0;
#pragma unroll 1
    for (int j = 0; j < q.units; j++) n += unit_cost(make_unit(b, q, j));
    return n;
}

// A place on the line: tile `off` of unit (request, head, j).
struct Place {
    int32_t req, head, unit, off;
};

// Quotients of the line's places.  Its length fits 32 bits but for very large batches, and a 64-bit
// division is a few hundred instructions of code that a short call would fetch for nothing else.
__device__ __forceinline__ long long line_div(long long a, long long b)
{
    if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
    return a / b;
}

// How the line is cut: part p of `used` takes the steps [total p / used, total (p + 1) / used).
struct Line {
    long long begin;  // this CTA's first step
    long long total;
    long long used;
    int steps;  // this CTA's; 0: none

    // The part that takes step x.
    __device__ __forceinline__ int part_of(long long x) const { return (int)line_div((x + 1) * used - 1, total); }
};

// Finds a CTA's piece of a line made of n_reqs stretches, the r-th cost(r) steps long; every thread of
// the block calls it.  scratch: one 8-byte word a warp.  Calls found(request, step inside its stretch) in
// the one thread that holds the piece's beginning.
template <int Threads, typename Cost, typename Found>
__device__ __forceinline__ Line find_piece(int n_reqs, int part, int parts, int least, long long *scratch, const Cost &cost, const Found &found)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int kWarps = Threads / 32;
    const int per = (n_reqs + Threads - 1) / Threads;
    const int r0 = min(tid * per, n_reqs), r1 = min(r0 + per, n_reqs);
    long long mine = 0;
#pragma unroll 1
    for (int r = r0; r < r1; r++) mine += cost(r);
    long long upto = mine;  // inclusive scan
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += o;
    }
    if (lane == 31) scratch[warp] = upto;
    __syncthreads();
    long long before = 0, total = 0;
#pragma unroll 1
    for (int w = 0; w < kWarps; w++) {
        if (w < warp) before += scratch[w];
        total += scratch[w];
    }
    upto += before;
    // pieces of at least `least` steps; none is empty but the last ones
    Line line{0, total, min((long long)parts, least == 1 ? total : line_div(total + least - 1, least)), 0};
    if (part < line.used) {
        line.begin = line_div(total * part, line.used);
        line.steps = (int)(line_div(total * (part + 1), line.used) - line.begin);
        if (line.begin >= upto - mine && line.begin < upto) {
            long long rest = line.begin - (upto - mine);
#pragma unroll 1
            for (int r = r0; r < r1; r++) {
                const long long all = r1 - r0 == 1 ? mine : cost(r);
                if (rest < all) {
                    found(r, rest);
                    break;
                }
                rest -= all;
            }
        }
    }
    __syncthreads();
    return line;
}

// This CTA's piece of an attention batch's line.
template <int Threads>
__device__ __forceinline__ Line find_place(const Batch &b, int part, int parts, int least, long long *scratch, Place *place, bool report)
{
    return find_piece<Threads>(
        b.n_reqs, part, parts, least, scratch, [&](int r) { return head_cost(b, load_request(b, r, report)) * b.kv_heads; },
        [&](int r, long long rest) {
            const Request q = load_request(b, r);
            const long long h = head_cost(b, q);
            Place p;
            p.req = r;
            p.head = (int)line_div(rest, h);
            rest -= p.head * h;
#pragma unroll 1
            for (p.unit = 0;; p.unit++) {
                const int n = unit_cost(make_unit(b, q, p.unit));
                if (rest < n) break;
                rest -= n;
            }
            p.off = (int)rest;
            *place = p;
        });
}

// Walks a piece unit by unit.
struct Walk {
    Place at;
    int left;
    Request q;
    Unit u;
    int n;  // tiles of the current fragment
    long long pos;  // its first step on the line

    __device__ __forceinline__ bool start(const Batch &b, const Place &p, const Line &line)
    {
        at = p;
        left = line.steps;
        pos = line.begin;
        if (left <= 0) return false;
        q = load_request(b, at.req);
        u = make_unit(b, q, at.unit);
        n = min(left, unit_cost(u) - at.off);
        return true;
    }
    // The fragment is the unit as a whole.
    __device__ __forceinline__ bool whole() const { return at.off == 0 && n == unit_cost(u); }
    __device__ __forceinline__ bool next(const Batch &b)
    {
        left -= n;
        pos += n;
        if (left <= 0) return false;
        at.off = 0;
        if (++at.unit == q.units) {
            at.unit = 0;
            if (++at.head == b.kv_heads) {
                at.head = 0;
                do {
                    q = load_request(b, ++at.req);
                } while (q.units == 0);  // `left` tiles remain, so a later request has rows
            }
        }
        u = make_unit(b, q, at.unit);
        n = min(left, unit_cost(u));
        return true;
    }
};

}  // namespace pkv
