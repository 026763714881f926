// How the attention kernels cut a ragged batch into work, on the device, from the lengths alone.
//
// A request's query rows are its (token, head of the group) pairs, token-major: row = token * group +
// head.  Rows are cut into units of `unit_rows`; a unit of one key head needs the key tiles of
// 2^tile_shift keys between the first key that its first token sees and the last that its last token sees.
// Laid end to end (request, key head, unit), all units' tiles form one line; CTA c of `parts` takes
// the c-th equal piece of it.  A piece may begin and end inside a unit: those two fragments go to the
// workspace, and whichever CTA finishes the unit's last one joins them.  So the split follows the
// lengths, not the launch: one grid serves a captured graph whatever the lengths become, and long
// contexts and few rows fill the GPU as well as many short requests do.
//
// A call of a few tiles a CTA spends most of its time fetching instructions that it runs once (about 40
// cycles each), so this code is kept short: 32-bit places, divisions by shifts and multiplications.
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
    int32_t tile_shift;
    int32_t causal;
    int32_t window;  // 0: none
    FastDiv group;   // query heads of a key head
    FastDiv unit;    // unit_rows
    int *err;
};

struct Request {
    int32_t q0, q_len, len;
    int32_t rows, units;
};

struct Unit {
    int32_t row0, rows;    // rows of the request
    int32_t lo, hi;        // keys that some row sees
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
    q.units = (int)fdiv((uint32_t)(q.rows + b.unit_rows - 1), b.unit);
    if (report && (a != q.q0 || e != end || (r == 0 && a != 0))) set_error(b.err, KV_DERR_LIST);
    if (report && n != q.len) set_error(b.err, KV_DERR_TABLE);
    return q;
}

// Keys [lo, hi) that query token t of the request sees.
__device__ __forceinline__ void sees(const Batch &b, const Request &q, int t, int &lo, int &hi)
{
    const int pos = q.len - q.q_len + t;
    hi = b.causal ? max(min(q.len, pos + 1), 0) : q.len;
    lo = b.window ? min(max(pos - b.window + 1, 0), hi) : 0;
}

__device__ __forceinline__ Unit make_unit(const Batch &b, const Request &q, int j)
{
    Unit u;
    u.row0 = j * b.unit_rows;
    u.rows = min(b.unit_rows, q.rows - u.row0);
    const int t0 = (int)fdiv((uint32_t)u.row0, b.group), t1 = (int)fdiv((uint32_t)(u.row0 + u.rows - 1), b.group);
    const int base = q.len - q.q_len;
    u.hi = b.causal ? max(min(q.len, base + t1 + 1), 0) : q.len;
    u.lo = b.window ? min(max(base + t0 - b.window + 1, 0), u.hi) : 0;
    u.tile0 = u.lo >> b.tile_shift;
    u.tiles = u.hi > u.lo ? ((u.hi - 1) >> b.tile_shift) + 1 - u.tile0 : 0;
    return u;
}

// A unit that sees nothing still takes one step of the line: its rows have to be written.
__device__ __forceinline__ int unit_cost(const Unit &u) { return max(1, u.tiles); }

__device__ __forceinline__ int head_cost(const Batch &b, const Request &q)
{
    int n = 0;
#pragma unroll 1
    for (int j = 0; j < q.units; j++) n += unit_cost(make_unit(b, q, j));
    return n;
}

// A place on the line: tile `off` of unit (request, head, j).
struct Place {
    int32_t req, head, unit, off;
};

// How the line of `total` steps is cut into parts: the first `more` of them take `each` + 1 steps, the
// others `each`.
struct Line {
    int32_t begin, steps;  // of this CTA's part; 0 steps: none
    int32_t each, more;

    __device__ __forceinline__ int part_of(int x) const  // the part that takes step x
    {
        const int longer = more * (each + 1);
        return x < longer ? (int)((uint32_t)x / (uint32_t)(each + 1)) : more + (int)((uint32_t)(x - longer) / (uint32_t)each);
    }
};

// Finds a CTA's piece of a line made of n_reqs stretches, the r-th cost(r) steps long (less than 2^31 in
// all); every thread of the block calls it.  Pieces are of at least `least` steps.  scratch: one word a
// warp.  Calls found(request, step inside its stretch) in the one thread that holds the beginning.
template <int Threads, typename Cost, typename Found>
__device__ __forceinline__ Line find_piece(int n_reqs, int part, int parts, int least, int *scratch, const Cost &cost, const Found &found)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (n_reqs + Threads - 1) / Threads;
    const int r0 = min(tid * per, n_reqs), r1 = min(r0 + per, n_reqs);
    int mine = 0;
#pragma unroll 1
    for (int r = r0; r < r1; r++) mine += cost(r);
    int upto = mine;  // inclusive scan
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += o;
    }
    if (lane == 31) scratch[warp] = upto;
    __syncthreads();
    int total = 0;
#pragma unroll 1
    for (int w = 0; w < Threads / 32; w++) {
        if (w == warp) upto += total;
        total += scratch[w];
    }
    // no part is empty but the last ones
    const int used = max(1, min(parts, least == 1 ? total : (total + least - 1) / least));
    Line line;
    line.each = (int)((uint32_t)total / (uint32_t)used);
    line.more = total - line.each * used;
    line.begin = part * line.each + min(part, line.more);
    line.steps = part < used ? line.each + (part < line.more) : 0;
    if (line.steps > 0 && line.begin >= upto - mine && line.begin < upto) {
        int rest = line.begin - (upto - mine);
#pragma unroll 1
        for (int r = r0; r < r1; r++) {
            const int all = r1 - r0 == 1 ? mine : cost(r);
            if (rest < all) {
                found(r, rest);
                break;
            }
            rest -= all;
        }
    }
    __syncthreads();
    return line;
}

// This CTA's piece of an attention batch's line.
template <int Threads>
__device__ __forceinline__ Line find_place(const Batch &b, int part, int parts, int least, int *scratch, Place *place, bool report)
{
    return find_piece<Threads>(
        b.n_reqs, part, parts, least, scratch, [&](int r) { return head_cost(b, load_request(b, r, report)) * b.kv_heads; },
        [&](int r, int rest) {
            const Request q = load_request(b, r);
            const int h = head_cost(b, q);
            Place p;
            p.req = r;
            p.head = (int)((uint32_t)rest / (uint32_t)h);
            rest -= p.head * h;
#pragma unroll 1
            for (p.unit = 0;; p.unit++) {
                const int n = unit_cost(make_unit(b, q, p.unit));
                if (rest < n) break;
                rest -= n;
            }
            p.off = rest;
            *place = p;
        });
}

// Walks a piece unit by unit.
struct Walk {
    Place at;
    int left;
    Request q;
    Unit u;
    int n;    // tiles of the current fragment
    int pos;  // its first step on the line

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
