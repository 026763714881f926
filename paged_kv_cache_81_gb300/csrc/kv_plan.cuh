// How the attention kernels cut a ragged batch into work, on the device, from the lengths alone.
//
// A request's query rows are its (token, head of the group) pairs, token-major: row = token * group +
// head.  Rows are cut into units of `unit_rows`; a unit of one key head needs the key tiles of
// 2^tile_shift keys between the first key that its first token sees and the last that its last token sees.
// Laid end to end (request, key head, unit), all units' tiles form one line; CTA c of `parts` takes
// the c-th equal piece of it.  A piece may begin and end inside a unit: those two fragments go to the
// workspace, and whichever CTA finishes the unit's last one joins them.  Where there are few units the
// pieces are cut unit by unit instead, so that none holds parts of two.  The split follows the
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

// Where a CTA's piece begins: step `off` of unit (request, head, unit).  nth: which of its unit's pieces this
// is, or -1 where the line is cut into equal pieces; steps: its length where it is not.
struct Place {
    int32_t req, head, unit, off, nth, steps;
};

// How the line is cut.  nth < 0: the first `more` parts take `each` + 1 steps, the others `each`.
// Otherwise every unit on its own into pieces of `each` steps.
struct Line {
    int32_t begin, steps;  // of this CTA's part; 0 steps: none
    int32_t each, more;
    int32_t part, nth;
    int32_t snap;  // an end of an equal piece this many steps from an edge of a unit, or fewer, moves there

    __device__ __forceinline__ int begin_of(int c) const { return c * each + min(c, more); }

    __device__ __forceinline__ int part_of(int x) const  // the part that takes step x of equal pieces
    {
        const int longer = more * (each + 1);
        return x < longer ? (int)((uint32_t)x / (uint32_t)(each + 1)) : more + (int)((uint32_t)(x - longer) / (uint32_t)each);
    }
};

__device__ __forceinline__ int ceil_div(int a, int b) { return (int)((uint32_t)(a + b - 1) / (uint32_t)b); }

// A thread's or warp's sum of steps, which stays at kTooLong once it gets there.  The hosts refuse batches whose steps
// would not fit 32 bits; offsets that decrease name requests that overlap, and many of those may add up to more.
constexpr int kTooLong = 0x7fffffff;
__device__ __forceinline__ int add_steps(int a, int b) { return (int)min((uint32_t)a + (uint32_t)b, (uint32_t)kTooLong); }

// Inclusive scan of `mine` over the block, and the sums of it and of `other`.  Where `mine` adds up to kTooLong or more, its sum
// is kTooLong or that of `other` negative (a sum that stopped there across the warps changed the code that uses it: a prompt of
// 32768 tokens under a window of 256 took 367 us instead of 361).  scratch: two words a warp.
template <int Threads>
__device__ __forceinline__ int block_scan(int mine, int other, int *scratch, int &total, int &other_total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int upto = mine;
#pragma unroll 1
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, upto, d);
        other += __shfl_xor_sync(0xffffffffu, other, d);
        if (lane >= d) upto = add_steps(upto, o);
    }
    if (lane == 31) scratch[2 * warp] = upto, scratch[2 * warp + 1] = other;
    __syncthreads();
    total = other_total = 0;
    int past = 0;
#pragma unroll 1
    for (int w = 0; w < Threads / 32; w++) {
        if (w == warp) upto = (int)((uint32_t)upto + (uint32_t)total);
        total = (int)((uint32_t)total + (uint32_t)scratch[2 * w]);
        past |= total;
        other_total += scratch[2 * w + 1];
    }
    other_total |= past & (int)0x80000000;
    return upto;
}

// Finds a CTA's piece; every thread of the block calls it.  The line is made of n_reqs stretches, and `work`
// says of one:
//   measure(r, steps, units)   adds its length (add_steps; less than 2^31) and its units
//   pieces(r, each)            its pieces when every unit is cut by itself into pieces of `each` steps
//   own(r, k, each)            the k-th of them (each = 1: step k)
// scratch: four words a warp.  Pieces of units are of at least `least` steps.  A line that is too long has no pieces.
//
// The ends of equal pieces move to the edge of a unit where that is within Work::kSnap steps (a cut costs both of its
// sides three or four), if pieces are long against that and units short enough for most ends to find an edge:
// 16 prompts of 1000 tokens, 16 heads of 128, 113 us without, 111 with 2 steps, 107 with 3; with keys of 192 129, 124
// and 121; units of 125 steps, whose cuts mostly stay, 185, 186 and 189.
//
// Units are cut by themselves when that makes the longest piece at most four steps longer: a piece that
// straddles two units pays twice for what a unit costs beside its tiles (queries, outputs, a join: 4 to 5
// us).  Eight latent requests of 200 to 2000 tokens, 16 heads: 23 us in equal pieces, 19 us so.
template <int Threads, typename Work>
__device__ __forceinline__ Line find_piece(int n_reqs, int part, int parts, int least, int *scratch, Place *place, const Work &work)
{
    const int per = n_reqs <= Threads ? 1 : ceil_div(n_reqs, Threads);
    const int r0 = min((int)threadIdx.x * per, n_reqs), r1 = min(r0 + per, n_reqs);
    int mine = 0, units = 0, total, unit_total;
#pragma unroll 1
    for (int r = r0; r < r1; r++) work.measure(r, mine, units);
    int at = block_scan<Threads>(mine, units, scratch, total, unit_total);
    if (total == kTooLong || unit_total < 0) total = 0, unit_total = 1 << 30;
    const int used = max(1, min(parts, total));
    Line line;
    line.part = part;
    line.nth = -1;
    line.snap = total / 32 <= unit_total && total >= 16 * used ? Work::kSnap : 0;
    line.each = (int)((uint32_t)total / (uint32_t)used);
    line.more = total - line.each * used;
    line.begin = part * line.each + min(part, line.more);
    line.steps = part < used ? line.each + (part < line.more) : 0;
    int target = line.begin, cut = 1;
    const int own = unit_total < parts ? max(least, ceil_div(total, parts - unit_total)) : 1 << 30;
    const bool by_unit = own <= max(least, line.each + 4);
    if (by_unit) {  // the same search over pieces instead of steps
        line.each = cut = own;
        line.snap = 0;
        target = part;
        mine = 0;
#pragma unroll 1
        for (int r = r0; r < r1; r++) mine += work.pieces(r, own);
        at = block_scan<Threads>(mine, 0, scratch + 2 * (Threads / 32), total, unit_total);
    }
    if (target < total && target >= at - mine && target < at) {
        int rest = target - (at - mine);
#pragma unroll 1
        for (int r = r0; r < r1; r++) {
            const int n = r1 - r0 == 1 ? mine : work.pieces(r, cut);
            if (rest < n) {
                *place = work.own(r, rest, cut);
                break;
            }
            rest -= n;
        }
    }
    __syncthreads();
    if (by_unit) {
        line.steps = part < total ? place->steps : 0;
        line.nth = place->nth;
    }
    return line;
}

// An attention batch's line.
struct AttentionWork {
    static constexpr int kSnap = 3;
    const Batch &b;
    bool report;
    __device__ __forceinline__ void measure(int r, int &steps, int &units) const
    {
        const Request q = load_request(b, r, report);
        steps = add_steps(steps, head_cost(b, q) * b.kv_heads);
        units += q.units * b.kv_heads;
    }
    __device__ __forceinline__ int head_pieces(const Request &q, int each) const
    {
        int n = 0;
#pragma unroll 1
        for (int j = 0; j < q.units; j++) n += ceil_div(unit_cost(make_unit(b, q, j)), each);
        return n;
    }
    __device__ __forceinline__ int pieces(int r, int each) const { return head_pieces(load_request(b, r), each) * b.kv_heads; }
    __device__ __forceinline__ Place own(int r, int k, int each) const
    {
        const Request q = load_request(b, r);
        const int h = head_pieces(q, each);
        Place p;
        p.req = r;
        p.head = (int)((uint32_t)k / (uint32_t)h);
        k -= p.head * h;
        int cost = 0;
#pragma unroll 1
        for (p.unit = 0;; p.unit++) {
            cost = unit_cost(make_unit(b, q, p.unit));
            const int n = ceil_div(cost, each);
            if (k < n) break;
            k -= n;
        }
        p.nth = k;
        p.off = k * each;
        p.steps = min(each, cost - p.off);
        return p;
    }
};

// This CTA's piece of it.
template <int Threads>
__device__ __forceinline__ Line find_place(const Batch &b, int part, int parts, int least, int *scratch, Place *place, bool report)
{
    return find_piece<Threads>(b.n_reqs, part, parts, least, scratch, place, AttentionWork{b, report});
}

// Walks a piece unit by unit.
struct Walk {
    Place at;
    int left;
    Request q;
    Unit u;
    int n;    // tiles of the current fragment
    int pos;  // its first step on the line
    int snap;

    __device__ __forceinline__ bool start(const Batch &b, const Place &p, const Line &line)
    {
        at = p;
        left = line.steps;
        pos = line.begin;
        snap = line.snap;
        if (left <= 0) return false;
        q = load_request(b, at.req);
        u = make_unit(b, q, at.unit);
        const int rest = unit_cost(u) - at.off;
        if (at.off <= snap && at.off <= rest) {
            left += at.off;
            pos -= at.off;
            at.off = 0;
        } else if (rest <= snap) {
            n = rest;
            return next(b);
        }
        return fit();
    }
    // What of the unit is this piece's; false if its end has moved to the unit's begin.
    __device__ __forceinline__ bool fit()
    {
        const int cost = unit_cost(u), end = at.off + left;
        if (end >= cost || (cost - end <= snap && cost - end < end))
            n = cost - at.off;
        else if (end <= snap)
            return false;
        else
            n = left;
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
        return fit();
    }
};

}  // namespace pkv
