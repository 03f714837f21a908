// attention_units.cuh -- how the many-rows attention kernel shares out its
// work: units of query rows, found from the lengths on the device, and the segments
// (units, or parts of units) that a thread block gets.  A whole warp calls all of
// it.  Nothing here but whole numbers and warp-wide exchanges, so that the tests can
// run it on the CPU.  (Included behind kv_cache.cuh.)
#pragma once

namespace qgemv {
namespace {

constexpr int kTile = 128;           // rows of a tile, entries of a step
constexpr int kUnitRows = 2 * kTile;
constexpr int kMaxBlocks = 160;  // as many as multiprocessors, at most
constexpr int kMinTiles = 2;    // entries' tiles of a part of a unit, at least
// What a unit costs besides its tiles, in tiles: queries, first scores, output
// (without it a block of 31 units of one tile counted as one of a unit of 31, and
// lasted four times as long).
constexpr int kUnitCost = 4;
// What cutting units costs, in tiles: two outputs in fp32, and their join.
constexpr int kSplitCost = 8;

// n / group by a multiplication: group_inv = floor(2^64 / group) + 1 (0 for 1).
__device__ __forceinline__ int div_group(const AttnArgs& a, int n) {
  return a.group == 1 ? n : static_cast<int>(__umul64hi(static_cast<unsigned long long>(n), a.group_inv));
}

// Finds a block's segments.  Units are ordered by sequence (up to 32 of them:
// the one with the longest units first), by row tile (the last, longest, first) and
// by head.  They go out in rounds of one per block: in the first as they come, so that
// the blocks that share keys stay next to one another, then the longest of a round
// to the block with the least so far (every scheduler works the whole table out, while
// the round before is computed; prompts of 1 to 4001 tokens, 384 units of 1 to 32 tiles:
// 88 us with rounds to and fro, 85 like this).  Or, with a workspace,
// the tiles of all units are cut into equal runs, one per block: a block's
// first and last unit may then be parts, whose results go to the workspace for the
// join.  Whichever is expected to be done sooner: whole units last as long as
// their rounds, or the longest of them, runs their length and kSplitCost.
// 2048 tokens over 30759 entries (256 units of 241 tiles for 152 blocks): whole
// 706 us, cut 660; 1200 over 9400 (152 units): whole 126, cut 143; 64 over 8064
// (8 units): whole 102, cut 29; the prompts above: whole 86, cut 95.
struct Scheduler {
  const AttnArgs& a;
  int lane;
  int s = -1, first = 0, count = 0, len = 0, rows = 0;  // sequence at hand,
  int place = 0;                                         // its place in the order
  int rt = 0, h = 0;                                     // unit at hand
  // Sequences s0 .. s0 + 31, one per lane: what they hold, their units, and the
  // spans of those (kUnitCost, then the tiles).
  int s0 = -1, c_id = 0, c_first = 0, c_count = 0, c_len = 0;
  long long c_units = 0, c_span = 0;
  int c_longest = 0;  // the longest span of one unit

  __device__ Scheduler(const AttnArgs& args, int l) : a(args), lane(l) {}

  __device__ static int units_of(int rows) { return (rows + kUnitRows - 1) / kUnitRows; }
  __device__ int rows_of(int n) const { return min(n, a.max_q) * a.group; }
  // tiles of entries that row tile r of a sequence sees, one at least
  __device__ int tiles_of(int r, int n_rows, int n_count, int n_len) const {
    const int last = min(n_rows, (r + 1) * kUnitRows) - 1;
    const int see = min(n_len, n_len - n_count + div_group(a, last) + 1);
    return max(1, (see + kTile - 1) / kTile);
  }
  // Take up the 32 sequences from i on.
  __device__ void look(int i, int* err) {
    if (s0 == i) return;
    s0 = i;
    c_first = c_count = c_len = 0;
    c_units = c_span = 0;
    c_longest = 0;
    if (i + lane < a.c.n_seqs) {
      seq_rows(a.q_start, i + lane, a.n_tokens, err, &c_first, &c_count);
      c_len = seq_len(a.c, i + lane, err);
      if (c_count > a.max_q) flag_error(err);
    }
    const int n_rows = rows_of(c_count), u = units_of(n_rows), n = min(32, a.c.n_seqs - i);
    c_units = static_cast<long long>(u) * a.c.n_kv;
    if (u > 0) c_longest = kUnitCost + tiles_of(u - 1, n_rows, c_count, c_len);
    if (n <= 16) {  // few sequences: their row tiles over the lanes
      for (int k = 0; k < n; ++k) {
        const int k_count = __shfl_sync(0xFFFFFFFFu, c_count, k), k_rows = rows_of(k_count);
        const int k_len = __shfl_sync(0xFFFFFFFFu, c_len, k), k_u = units_of(k_rows);
        // 32 bits where they are enough: the start of every call waits for this
        if (static_cast<long long>(k_u) * (kUnitCost + k_len / kTile + 1) <= 0x7FFFFFFF) {
          int t = 0;
          for (int r = lane; r < k_u; r += 32) t += kUnitCost + tiles_of(r, k_rows, k_count, k_len);
          t = __reduce_add_sync(0xFFFFFFFFu, t);
          if (lane == k) c_span = t;
          continue;
        }
        long long t = 0;  // (2^22 row tiles of up to 2^22 tiles, a lane has less than 2^40)
        for (int r = lane; r < k_u; r += 32) t += kUnitCost + tiles_of(r, k_rows, k_count, k_len);
        const unsigned lo = __reduce_add_sync(0xFFFFFFFFu, static_cast<unsigned>(t & 0x3FFFFFF));
        const unsigned hi = __reduce_add_sync(0xFFFFFFFFu, static_cast<unsigned>(t >> 26));
        if (lane == k) c_span = (static_cast<long long>(hi) << 26) + lo;
      }
    } else {
      for (int r = 0; r < u; ++r) c_span += kUnitCost + tiles_of(r, n_rows, c_count, c_len);
    }
    c_span *= a.c.n_kv;
    c_id = i + lane;
    if (a.c.n_seqs > 1 && a.c.n_seqs <= 32) {  // those with the longest units first
      int rank = 0;
      for (int k = 0; k < a.c.n_seqs; ++k) {
        const int other = __shfl_sync(0xFFFFFFFFu, c_longest, k);
        rank += other > c_longest || (other == c_longest && k < lane);
      }
      int from = 0;  // the lane whose rank is this lane's number
      for (int k = 0; k < a.c.n_seqs; ++k)
        if (__shfl_sync(0xFFFFFFFFu, rank, k) == lane) from = k;
      c_id = __shfl_sync(0xFFFFFFFFu, c_id, from);
      c_first = __shfl_sync(0xFFFFFFFFu, c_first, from);
      c_count = __shfl_sync(0xFFFFFFFFu, c_count, from);
      c_len = __shfl_sync(0xFFFFFFFFu, c_len, from);
      c_units = __shfl_sync(0xFFFFFFFFu, c_units, from);
      c_span = __shfl_sync(0xFFFFFFFFu, c_span, from);
      c_longest = __shfl_sync(0xFFFFFFFFu, c_longest, from);
      if (lane >= a.c.n_seqs) c_units = c_span = c_longest = 0;  // (nobody's rank)
    }
  }
  __device__ void total(int* err, long long* units, long long* span, int* longest) {
    long long n = 0, t = 0;
    int m = 0;
    for (int i = 0; i < a.c.n_seqs; i += 32) {
      look(i, err);
      n += c_units;
      t += c_span;
      m = max(m, c_longest);
    }
#pragma unroll
    for (int k = 16; k > 0; k /= 2) {
      n += __shfl_xor_sync(0xFFFFFFFFu, n, k);
      t += __shfl_xor_sync(0xFFFFFFFFu, t, k);
    }
    *units = n;
    *span = t;
    *longest = __reduce_max_sync(0xFFFFFFFFu, m);
  }
  __device__ static long long scan(long long v, int lane) {
#pragma unroll
    for (int k = 1; k < 32; k *= 2) {
      const long long w = __shfl_up_sync(0xFFFFFFFFu, v, k);
      if (lane >= k) v += w;
    }
    return v;
  }
  // Go to the unit that holds position pos of all spans (of all units, one
  // each); the position within it, or -1 if there is none.
  __device__ int seek(long long pos, bool spans) {
    for (int i = 0; i < a.c.n_seqs; i += 32) {
      look(i, nullptr);
      const long long mine = spans ? c_span : c_units, incl = scan(mine, lane);
      const unsigned hit = __ballot_sync(0xFFFFFFFFu, pos < incl);
      if (hit == 0) {
        pos -= __shfl_sync(0xFFFFFFFFu, incl, 31);
        continue;
      }
      const int l = __ffs(hit) - 1;
      pos -= __shfl_sync(0xFFFFFFFFu, incl - mine, l);
      place = i + l;
      s = __shfl_sync(0xFFFFFFFFu, c_id, l);
      first = __shfl_sync(0xFFFFFFFFu, c_first, l);
      count = __shfl_sync(0xFFFFFFFFu, c_count, l);
      len = __shfl_sync(0xFFFFFFFFu, c_len, l);
      rows = rows_of(count);
      for (int top = units_of(rows) - 1; top >= 0; top -= 32) {
        const int r = top - lane;  // this lane's row tile
        const int each = r < 0 ? 0 : spans ? kUnitCost + tiles_of(r, rows, count, len) : 1;
        const long long here = static_cast<long long>(each) * a.c.n_kv, to = scan(here, lane);
        const unsigned in = __ballot_sync(0xFFFFFFFFu, pos < to);
        if (in == 0) {
          pos -= __shfl_sync(0xFFFFFFFFu, to, 31);
          continue;
        }
        const int k = __ffs(in) - 1;
        long long rest = pos - __shfl_sync(0xFFFFFFFFu, to - here, k);
        const int step = __shfl_sync(0xFFFFFFFFu, each, k);
        rt = top - k;
        h = 0;
        if (rest >> 31 != 0) {  // (1024 heads of 2^22 + 4 at most: below 2^32 without half of them)
          h = a.c.n_kv / 2;
          rest -= static_cast<long long>(h) * step;
        }
        const unsigned left = static_cast<unsigned>(rest);
        h += left / step;
        return left % step;
      }
    }
    return -1;
  }
  // A unit to come back to.
  struct Mark {
    int s, first, count, len, rows, place, rt, h;
  };
  __device__ Mark mark() const { return {s, first, count, len, rows, place, rt, h}; }
  __device__ void back(const Mark& m) {
    s = m.s, first = m.first, count = m.count, len = m.len;
    rows = m.rows, place = m.place, rt = m.rt, h = m.h;
  }
  // The unit n units on; false behind the last.
  __device__ bool advance(int n) {
    h += n;
    while (h >= a.c.n_kv) {
      h -= a.c.n_kv;
      while (--rt < 0) {
        if (++place >= a.c.n_seqs) return false;
        look(place & ~31, nullptr);
        const int l = place & 31;
        s = __shfl_sync(0xFFFFFFFFu, c_id, l);
        first = __shfl_sync(0xFFFFFFFFu, c_first, l);
        count = __shfl_sync(0xFFFFFFFFu, c_count, l);
        len = __shfl_sync(0xFFFFFFFFu, c_len, l);
        rows = rows_of(count);
        rt = units_of(rows);
      }
    }
    return true;
  }
};

// Hands this block's segments to emit(end, j0, j1, slot), with the unit in sc; the
// unit of which this block has the first part, but not all, is the answer.  s_span,
// s_load, s_order: kMaxBlocks elements each, in shared memory.  (emit by reference: as a
// copy, what it refers to, and with it the scheduler, was kept in local memory.)
template <typename Emit>
__device__ __forceinline__ AttnUnit hand_out(const AttnArgs& a, Scheduler& sc, int lane, int* s_span,
                                             int* s_load, uint8_t* s_order, Emit& emit) {
  int* err = blockIdx.x == 0 ? a.err : nullptr;
  long long units, all;
  int longest;
  sc.total(err, &units, &all, &longest);
  const long long rounds = (units + gridDim.x - 1) / gridDim.x;
  const long long whole = max(static_cast<long long>(longest), rounds * all / max(1LL, units));
  const long long per = max(static_cast<long long>(kUnitCost + kMinTiles),
                            (all + gridDim.x - 1) / gridDim.x);
  AttnUnit split{};
  if (a.splits != nullptr && per + kSplitCost < whole) {
    long long left = min(per, all - blockIdx.x * per);
    if (left > 0) {
      int p0 = sc.seek(blockIdx.x * per, true);  // place in the unit's span
      bool more = p0 >= 0;
      while (more) {
        const int t = sc.tiles_of(sc.rt, sc.rows, sc.count, sc.len);
        const int p1 = static_cast<int>(min(static_cast<long long>(kUnitCost + t), p0 + left));
        const int j0 = max(0, p0 - kUnitCost), j1 = max(0, p1 - kUnitCost);
        if (j1 > j0) {
          if (j0 == 0 && j1 < t)
            split = AttnUnit{1 + static_cast<int>((t - j1 + per - 1) / per), sc.s, sc.h,
                             sc.rt * kUnitRows, sc.first, sc.rows, sc.len - sc.count, sc.len};
          emit(false, j0, j1,
               j0 > 0 || j1 < t ? 2 * static_cast<int>(blockIdx.x) + (j0 == 0) : -1);
        }
        left -= p1 - p0;
        p0 = 0;
        more = left > 0 && sc.advance(1);
      }
    }
  } else if (units > 0 && sc.seek(0, false) >= 0) {
    constexpr int kOwn = kMaxBlocks / 32;
    const int blocks = gridDim.x, me = blockIdx.x;
    auto emit_unit = [&](int n) {  // the n-th from here
      if (sc.advance(n)) emit(false, 0, sc.tiles_of(sc.rt, sc.rows, sc.count, sc.len), -1);
    };
    int load[kOwn] = {};  // of blocks lane, lane + 32 ..
    bool more = true;
    for (long long at = 0; more; at += blocks) {
      const int n = static_cast<int>(min(static_cast<long long>(blocks), units - at));
      const auto start = sc.mark();
      if (at == 0) {
        if (me < n) emit_unit(me);
        if (units <= blocks) break;
        sc.back(start);
      }
      for (int i = 0; i < n;) {  // the spans of the round's units
        const int run = min(n - i, a.c.n_kv - sc.h);
        const int t = kUnitCost + sc.tiles_of(sc.rt, sc.rows, sc.count, sc.len);
        for (int k = i + lane; k < i + run; k += 32) s_span[k] = t;
        i += run;
        more = sc.advance(run);
      }
      const auto end = sc.mark();
#pragma unroll
      for (int u = 0; u < kOwn; ++u) s_load[lane + 32 * u] = load[u];
      __syncwarp();
      int rank[kOwn] = {}, own[kOwn];  // of this lane's units, longest first
#pragma unroll
      for (int u = 0; u < kOwn; ++u) own[u] = lane + 32 * u < n ? s_span[lane + 32 * u] : 0;
      for (int k = 0; k < n; ++k) {
        const int t = s_span[k];
#pragma unroll
        for (int u = 0; u < kOwn; ++u) rank[u] += t > own[u] || (t == own[u] && k < lane + 32 * u);
      }
#pragma unroll
      for (int u = 0; u < kOwn; ++u)
        if (lane + 32 * u < n) s_order[at == 0 ? lane + 32 * u : rank[u]] = lane + 32 * u;
      __syncwarp();
#pragma unroll
      for (int u = 0; u < kOwn; ++u) rank[u] = 0;  // of this lane's blocks, least first
      for (int k = 0; k < blocks; ++k) {
        const int t = s_load[k];
#pragma unroll
        for (int u = 0; u < kOwn; ++u) rank[u] += t < load[u] || (t == load[u] && k < lane + 32 * u);
      }
      int mine = -1;  // the round's unit that this block takes
#pragma unroll
      for (int u = 0; u < kOwn; ++u) {
        const int unit = lane + 32 * u < blocks && rank[u] < n ? s_order[rank[u]] : -1;
        if (unit >= 0) load[u] += s_span[unit];
        const int found = __shfl_sync(0xFFFFFFFFu, unit, me % 32);
        if (u == me / 32) mine = found;
      }
      __syncwarp();  // the next round's spans and loads take these ones' place
      if (at > 0 && mine >= 0) {
        sc.back(start);
        emit_unit(mine);
        sc.back(end);
      }
    }
  }
  return split;
}

}  // namespace
}  // namespace qgemv
