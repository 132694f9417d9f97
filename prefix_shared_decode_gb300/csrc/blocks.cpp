// Schedules of query blocks: which tile of which block's rows reads which of
// its context's chunks.
//
// A block's rows of one key/value head (query tokens x heads of the group) are
// cut into tiles; a tile reads the chunks that any of its rows may see.  Every
// place on the card gets a list of tiles, or of pieces of tiles along their
// chunks, which are joined afterwards.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <functional>
#include <numeric>

#include "ca_internal.h"

namespace ca {

namespace {
size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
// A piece of a tile's chunks holds at least this many tokens (its queries are
// read, and its partial written and joined, whatever it holds); the tokens of a
// step of the kernels; what an item costs whatever it reads, in tokens, and the
// joining of pieces in a kernel of its own; and what a token costs a tile that
// fills half of its rows at most.  From traced times of items over fp16 pools at 128
// dims (a step of 128 tokens some 1.8 us, an item's start and end 3, a join 5 to 8),
// and taken for the other dims and pools too: a choice that they make badly costs
// time alone.  With them 32 tiles over 16384 tokens each are cut (52 us; each into
// equal pieces, 160 of them on 152 places, 80), and 448 tiles at 64 dims over some
// 1220 tokens are not (64 us when it was measured, cut 76).
constexpr int32_t kPieceTokens = 256, kStepTokens = 128;
constexpr double kItemCost = 200, kJoinCost = 500, kHalfTileCost = 0.6;
}  // namespace

int build_blocks(const Pool& p, const int64_t* seq_ids, int32_t b, const int32_t* q_lens, uint32_t flags, Sched& s) {
    const int32_t c = p.cfg.chunk, HK = kv_heads(p.cfg), G = p.cfg.n_heads / HK, T = cross_tile_rows(p.cfg);
    const bool causal = (flags & CA_SCHED_CAUSAL) != 0;
    std::vector<const Sequence*> seq(b);
    int64_t rows = 0, chunks = 0, n_tiles = 0;
    for (int32_t i = 0; i < b; ++i) {
        auto it = p.seqs.find(seq_ids[i]);
        if (it == p.seqs.end()) return CA_ERR_NOT_FOUND;
        if (q_lens[i] < 0) return CA_ERR_INVALID;
        seq[i] = &it->second;
        rows += q_lens[i];
        chunks += (int64_t)it->second.path.size();
        if ((int64_t)q_lens[i] * G > INT32_MAX - T) return CA_ERR_UNSUPPORTED;
        n_tiles += ((int64_t)q_lens[i] * G + T - 1) / T;
    }
    if (rows > INT32_MAX || chunks > INT32_MAX || n_tiles * HK > INT32_MAX / 64) return CA_ERR_UNSUPPORTED;

    // Tiles of each sequence's rows, and the chunks that each one reads.
    struct Tile { int32_t seq, row0, rows, chunks; };
    std::vector<Tile> tiles;
    std::vector<int32_t> first_tile(1, 0), list0(1, 0), q_off(1, 0);
    auto cost = [T](const Tile& t) { return t.rows <= T / 2 && T > 128 ? kHalfTileCost : 1.0; };   // of a token
    double total = 0;
    for (int32_t i = 0; i < b; ++i) {
        const int32_t n = seq[i]->length, m = q_lens[i], R = m * G;
        for (int32_t r = 0; r < R; r += T) {
            const int32_t take = std::min(T, R - r);
            // (without a mask the last chunk may grow in place: all chunks)
            const int32_t seen = causal ? std::max(0, n - m + (r + take - 1) / G + 1) : n;
            tiles.push_back({i, r, take, (seen + c - 1) / c});
            total += HK * (kItemCost + cost(tiles.back()) * tiles.back().chunks * c);
        }
        first_tile.push_back((int32_t)tiles.size());
        list0.push_back(list0.back() + (int32_t)seq[i]->path.size());
        q_off.push_back(q_off.back() + q_lens[i]);
    }

    // Every place on the card gets a list of items.  Either whole tiles, the
    // longest first, each to the place with least work so far; or, where that
    // leaves places idle for longer than joining takes, all tiles behind one another
    // are cut into equal stretches.
    const int64_t most = std::max(1, cross_places(p));
    std::vector<BlockItem> items;
    std::vector<BlockJoin> joins;
    std::vector<int32_t> begin(1, 0);                       // of each place's items
    int64_t parts = 0;
    auto item = [&](const Tile& t, int32_t h, int32_t from, int32_t to) {
        items.push_back({t.seq, h, t.row0, t.rows, from, to, -1, q_off[t.seq], q_lens[t.seq], seq[t.seq]->length,
                         (int32_t)seq[t.seq]->path.size(), list0[t.seq], seq[t.seq]->path.back()->slot, {0, 0, 0}});
    };
    auto tile_cost = [&](const Tile& t) { return kItemCost + cost(t) * t.chunks * c; };

    std::vector<int32_t> order(tiles.size() * HK);          // tile * HK + head, by falling cost
    std::iota(order.begin(), order.end(), 0);
    std::stable_sort(order.begin(), order.end(),
                     [&](int32_t x, int32_t y) { return tile_cost(tiles[x / HK]) > tile_cost(tiles[y / HK]); });
    const int64_t n_whole = std::min<int64_t>(most, std::max<int64_t>(1, (int64_t)order.size()));
    std::vector<std::pair<double, int32_t>> load(n_whole);  // a heap, least work on top
    for (int64_t k = 0; k < n_whole; ++k) load[k] = {0.0, (int32_t)k};
    std::vector<int32_t> place_of(order.size());
    double longest = 0;
    for (size_t k = 0; k < order.size(); ++k) {
        std::pop_heap(load.begin(), load.end(), std::greater<>());
        load.back().first += tile_cost(tiles[order[k] / HK]);
        place_of[k] = load.back().second;
        longest = std::max(longest, load.back().first);
        std::push_heap(load.begin(), load.end(), std::greater<>());
    }
    const double share = std::max(total / most, kItemCost + kPieceTokens);
    int64_t n_places = n_whole;
    if (longest <= share + kItemCost + kJoinCost) {
        std::vector<int32_t> count(n_whole + 1, 0);
        for (int32_t k : place_of) ++count[k + 1];
        for (int64_t k = 0; k < n_whole; ++k) count[k + 1] += count[k];
        begin = count;
        std::vector<int32_t> sorted(order.size());
        for (size_t k = 0; k < order.size(); ++k) sorted[count[place_of[k]]++] = order[k];
        for (int32_t k : sorted) item(tiles[k / HK], k % HK, 0, tiles[k / HK].chunks);
    } else {
        // A cut falls on a whole step of the kernels, and on a tile's end where it
        // would leave a piece of fewer than kPieceTokens.
        n_places = std::clamp<int64_t>((int64_t)std::ceil(total / share), 1, most);   // (the quotient may round up)
        const int32_t grain = std::max(1, kStepTokens / c), least = std::max(1, kPieceTokens / c);
        double x = 0;
        auto next_cut = [&] { return (double)begin.size() * share; };
        for (int32_t i = 0; i < b; ++i)
            for (int32_t h = 0; h < HK; ++h)
                for (int32_t k = first_tile[i]; k < first_tile[i + 1]; ++k) {
                    const Tile& t = tiles[k];
                    const double per = cost(t) * c, end = x + tile_cost(t);
                    const size_t first = items.size();
                    int32_t at = 0;
                    while ((int64_t)begin.size() < n_places && next_cut() < end) {
                        const int32_t cut = (int32_t)((next_cut() - x - kItemCost) / per / grain + 0.5) * grain;
                        if (t.chunks - cut < least) break;  // behind the tile
                        if (cut - at >= least) {
                            item(t, h, at, cut);
                            at = cut;
                        }
                        begin.push_back((int32_t)items.size());
                    }
                    item(t, h, at, t.chunks);
                    while ((int64_t)begin.size() < n_places && next_cut() < end) begin.push_back((int32_t)items.size());
                    x = end;
                    const int64_t n = (int64_t)(items.size() - first);
                    if (n > 1) {
                        if (parts + n > INT32_MAX / 2) return CA_ERR_UNSUPPORTED;
                        joins.push_back({i, h, t.row0, t.rows, (int32_t)parts, (int32_t)n, 0, 0});
                        for (size_t y = first; y < items.size(); ++y) items[y].part = (int32_t)parts++;
                    }
                }
        begin.resize((size_t)n_places, (int32_t)items.size());
        begin.push_back((int32_t)items.size());
    }

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
    s.n_places = (int32_t)n_places;

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
    place(lay.cta_begin, begin.size() * sizeof(int32_t));
    place(lay.joins, s.joins.size() * sizeof(BlockJoin));
    lay.total = off;
    s.blob.assign(off, 0);
    auto put = [&s](size_t at, const void* src, size_t bytes) {
        if (bytes) std::memcpy(s.blob.data() + at, src, bytes);
    };
    put(lay.list_slots, s.t.list_slots.data(), s.t.list_slots.size() * sizeof(int32_t));
    put(lay.q_off, q_off.data(), q_off.size() * sizeof(int32_t));
    put(lay.items, s.items.data(), s.items.size() * sizeof(BlockItem));
    put(lay.cta_begin, begin.data(), begin.size() * sizeof(int32_t));
    put(lay.joins, s.joins.data(), s.joins.size() * sizeof(BlockJoin));

    s.ws = WsLayout{};
    const size_t D = p.cfg.head_dim;
    s.ws.part_o = 0;
    s.ws.part_ms = align256((size_t)parts * T * D * sizeof(float));
    s.ws.total = s.ws.part_ms + align256((size_t)parts * T * 2 * sizeof(float));
    return CA_OK;
}

}  // namespace ca
