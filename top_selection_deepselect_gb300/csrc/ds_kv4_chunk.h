// ds_kv4_chunk.h -- how attention of chunks is laid out: what the planning launch,
// the kernels and the host share.
#pragma once

#include "ds_kv4.cuh"
#include "ds_kv4_launch.h"

namespace ds {
namespace kv4 {
namespace chunk {

// Tiles of 128 query rows of a block: two, unless their outputs leave no room in
// tensor memory.
constexpr int tiles_of_rows(int d) { return d == 256 ? 1 : 2; }

// A block of rows of one batch entry: rows [row0, row0 + Args::rows) of its n * group.
struct alignas(16) Block {
    long long place;      // places of the line, for one head, before it
    int seq, start, n;    // the sequence, its first row of q, its new tokens
    int len, row0, pad;
};

struct Head {
    long long all, per;   // places of the line, of a CTA
    int blocks, pad;
};

// Left for the join: the unit that begins in a CTA and goes on in others.
struct alignas(16) Split {
    int block, head, parts, pad;
};

struct Args {
    Cache c;
    Chunk a;
    Head *head;
    Block *blocks;
    int *first;           // block that a CTA's first place is in
    Split *splits;
    float *partial;
    int group, rows, run, ctas, q_vector;
    int few;              // few blocks and little work: each CTA lays them out itself, without the
                          // planning launch
    int whole;            // short sequences: units are not cut, and there is nothing to join
    Divider by_group;
};

// Entries and blocks that a warp lays out, a lane each.
constexpr int kFew = 32;
// Places of a CTA where units are cut: not more parts to join than the work is worth.
constexpr int kLeast = 96;

// What is known of entry b: its sequence and length; start and n are left to the caller.
struct Entry {
    int seq, start, n, len;
};
__device__ __forceinline__ Entry entry_of(const Args &p, int b)
{
    Entry e;
    e.seq = p.a.seqs ? p.a.seqs[b] : b;
    e.start = e.n = e.len = 0;
    if ((unsigned)e.seq < (unsigned)p.c.max_seqs) {
        const int n = p.a.lengths[e.seq];
        const long long room = (long long)p.c.max_pages * p.c.page_size;
        e.len = n < 0 ? 0 : n > room ? (int)room : n;
    }
    return e;
}
__device__ __forceinline__ int start_of(const Args &p, int b)      // of entry b, within the rows
{
    const int x = p.a.starts[b];
    return x < 0 ? 0 : x > p.a.tokens ? p.a.tokens : x;
}
__device__ __forceinline__ long long places_of_cta(const Args &p, long long all)
{
    const long long even = (all + p.ctas - 1) / p.ctas;
    return p.whole || even > kLeast ? (even > 1 ? even : 1) : kLeast;
}

// What a block's rows see, and its tiles.
struct Span {
    int rows, row_tiles, see_lo, see_hi, tiles;
    int weight;           // places of a tile
};

__device__ __forceinline__ Span span_of(const Block &b, const Divider &by_group, int group, int block_rows)
{
    Span s;
    const int left = b.n * group - b.row0;
    s.rows = left < block_rows ? left : block_rows;
    s.row_tiles = s.rows > 128 ? 2 : 1;
    const int lo = b.len - b.n + 1 + by_group(b.row0), hi = b.len - b.n + 1 + by_group(b.row0 + s.rows - 1);
    s.see_lo = lo > 0 ? lo : 0;
    s.see_hi = hi > 0 ? hi : 0;
    s.tiles = s.see_hi / 64 + (s.see_hi % 64 != 0);
    // A rule from 2 x 129 tokens after 130943 with heads of 128, of whose rows one block in
    // five is small: 1232 us, with 6 1290 and with 8 1274.  With heads of 64 8 is better
    // (1108 and 1061), of 256 there is one row tile a block anyhow.
    s.weight = s.row_tiles == 2 ? 8 : 7;
    return s;
}

// Places of a unit: of its tiles, and of its start and end (queries, first copies,
// outputs), by what they take: ragged prompts of 9 x 701 tokens at most, heads of 64, fp16
// 176 us with 40, 196 with 16, 180 with 64; bf16 160, 176 and 154; of 128 bf16 203, 224 and
// 186; of 256 bf16 412, 484 and 420.  One number for all, at most 9 % off the better one.
constexpr int kUnitCost = 40;
__device__ __forceinline__ int cost_of(const Span &s) { return kUnitCost + s.tiles * s.weight; }

}  // namespace chunk
}  // namespace kv4
}  // namespace ds
