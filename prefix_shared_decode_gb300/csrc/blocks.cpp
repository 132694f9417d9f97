// Schedules of query blocks: which tile of which block's rows reads which of
// its context's chunks.
//
// A block's rows of one key/value head (query tokens x heads of the group) are
// cut into tiles; a tile reads the chunks that any of its rows may see.  Where a
// batch has fewer tiles than the card has places for, the longer ones are cut
// along their chunks too and joined afterwards.  Items are listed by falling
// length, so that the last ones to run are short.
#include <algorithm>
#include <cstring>

#include "ca_internal.h"

namespace ca {

namespace {
size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
// A piece of a tile's chunks holds at least this many tokens (its queries are
// read, and its partial written and joined, whatever it holds).
constexpr int32_t kPieceTokens = 256;
}  // namespace

int build_blocks(const Pool& p, const int64_t* seq_ids, int32_t b, const int32_t* q_lens, uint32_t flags, Sched& s) {
    const int32_t c = p.cfg.chunk, HK = kv_heads(p.cfg), G = p.cfg.n_heads / HK, T = cross_tile_rows(p.cfg);
    const bool causal = (flags & CA_SCHED_CAUSAL) != 0;
    std::vector<const Sequence*> seq(b);
    int64_t rows = 0, chunks = 0;
    for (int32_t i = 0; i < b; ++i) {
        auto it = p.seqs.find(seq_ids[i]);
        if (it == p.seqs.end()) return CA_ERR_NOT_FOUND;
        if (q_lens[i] < 0) return CA_ERR_INVALID;
        seq[i] = &it->second;
        rows += q_lens[i];
        chunks += (int64_t)it->second.path.size();
        if ((int64_t)q_lens[i] * G > INT32_MAX - T) return CA_ERR_UNSUPPORTED;
    }
    if (rows > INT32_MAX || chunks > INT32_MAX) return CA_ERR_UNSUPPORTED;

    // Tiles, and the tokens that each one reads.
    struct Tile { int32_t seq, row0, rows, chunks; };
    std::vector<Tile> tiles;
    int64_t total = 0;                  // chunks that all of a head's tiles read
    for (int32_t i = 0; i < b; ++i) {
        const int32_t n = seq[i]->length, m = q_lens[i], R = m * G;
        for (int32_t r = 0; r < R; r += T) {
            const int32_t take = std::min(T, R - r);
            // (without a mask the last chunk may grow in place: all chunks)
            const int32_t seen = causal ? std::max(0, n - m + (r + take - 1) / G + 1) : n;
            const int32_t k = (seen + c - 1) / c;
            tiles.push_back({i, r, take, k});
            total += k;
        }
    }
    if ((int64_t)tiles.size() * HK > INT32_MAX / 64) return CA_ERR_UNSUPPORTED;

    // Pieces: of the average load of a place on the card, where a tile is longer.
    const int64_t places = std::max(1, cross_places(p));
    const int64_t per = std::max<int64_t>(std::max(1, kPieceTokens / c), (total * HK + places - 1) / places);
    std::vector<BlockItem> items;
    std::vector<BlockJoin> joins;
    int64_t parts = 0;
    std::vector<int32_t> list0(1, 0), q_off(1, 0);
    for (int32_t i = 0; i < b; ++i) {
        list0.push_back(list0.back() + (int32_t)seq[i]->path.size());
        q_off.push_back(q_off.back() + q_lens[i]);
    }
    for (const Tile& t : tiles) {
        const Sequence& of = *seq[t.seq];
        const int64_t n = std::max<int64_t>(1, (t.chunks + per - 1) / per);
        for (int32_t h = 0; h < HK; ++h) {
            if (n > 1) joins.push_back({t.seq, h, t.row0, t.rows, (int32_t)parts, (int32_t)n, 0, 0});
            for (int64_t x = 0; x < n; ++x)
                items.push_back({t.seq, h, t.row0, t.rows, (int32_t)(t.chunks * x / n), (int32_t)(t.chunks * (x + 1) / n),
                                 n > 1 ? (int32_t)parts++ : -1, q_off[t.seq], q_lens[t.seq], of.length,
                                 (int32_t)of.path.size(), list0[t.seq], of.path.back()->slot, {0, 0, 0}});
        }
        if (parts > INT32_MAX / 2) return CA_ERR_UNSUPPORTED;
    }
    std::stable_sort(items.begin(), items.end(), [](const BlockItem& x, const BlockItem& y) {
        return x.c_end - x.c_begin > y.c_end - y.c_begin;
    });

    // The schedule's tables (nothing above has changed it).
    s.t = Tables{};
    s.plan = Plan{};
    s.t.b = b;
    for (int32_t i = 0; i < b; ++i) {
        for (const Node* x : seq[i]->path) s.t.list_slots.push_back(x->slot);
        s.t.ctx_len.push_back(seq[i]->length);
    }
    s.q_lens.assign(q_lens, q_lens + b);
    s.q_rows = rows;
    s.items = std::move(items);
    s.joins = std::move(joins);
    s.n_parts = (int32_t)parts;
    s.tile_rows = T;

    PlanLayout& lay = s.layout;
    lay = PlanLayout{};
    size_t off = 0;
    auto place = [&off](size_t& at, size_t bytes) {
        at = off;
        off = align256(off + bytes);
    };
    place(lay.status, sizeof(int32_t));
    place(lay.counter, sizeof(int32_t));
    place(lay.list_count, 0);
    place(lay.list_slots, s.t.list_slots.size() * sizeof(int32_t));
    place(lay.q_off, q_off.size() * sizeof(int32_t));
    place(lay.items, s.items.size() * sizeof(BlockItem));
    place(lay.joins, s.joins.size() * sizeof(BlockJoin));
    lay.total = off;
    s.blob.assign(off, 0);
    auto put = [&s](size_t at, const void* src, size_t bytes) {
        if (bytes) std::memcpy(s.blob.data() + at, src, bytes);
    };
    put(lay.list_slots, s.t.list_slots.data(), s.t.list_slots.size() * sizeof(int32_t));
    put(lay.q_off, q_off.data(), q_off.size() * sizeof(int32_t));
    put(lay.items, s.items.data(), s.items.size() * sizeof(BlockItem));
    put(lay.joins, s.joins.data(), s.joins.size() * sizeof(BlockJoin));

    s.ws = WsLayout{};
    const size_t D = p.cfg.head_dim;
    s.ws.part_o = 0;
    s.ws.part_ms = align256((size_t)parts * T * D * sizeof(float));
    s.ws.total = s.ws.part_ms + align256((size_t)parts * T * 2 * sizeof(float));
    s.ws.total_host = s.ws.weights_total = s.ws.total;
    return CA_OK;
}

}  // namespace ca
