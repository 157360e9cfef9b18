// train_schedule.cpp -- the training products' schedule (csrc/tg_plan.h), walked
// on the CPU for tests/test_train_schedule.py: what the kernels' workers do, from
// the same functions, checked for covering every k step of every tile once, for
// places within the buffers, and for joins that add just the parts that were
// stored.  Every check returns "" or what is wrong.
#include <cstdio>
#include <cstring>
#include <map>
#include <set>
#include <string>
#include <tuple>
#include <vector>

#include "launch.h"
#include "tg_plan.h"

using namespace fmca;

namespace {

using Tile = std::tuple<int, int, int>;  // problem, row tile, column tile

#define FAIL(...)                              \
  do {                                         \
    char text[256];                            \
    std::snprintf(text, sizeof(text), __VA_ARGS__); \
    return std::string(text);                  \
  } while (0)

struct Stored {
  int k0, n, part;
};
using Parts = std::map<Tile, std::vector<Stored>>;

// A piece's units: every k step of every tile that exists once, at most two cut
// tiles a worker.
template <int CG, int KIND, int NT>
std::string walk_piece(const TgPlan &p, int W, Parts &parts) {
  std::map<Tile, std::vector<std::pair<int, int>>> steps;
  std::set<int> used;
  for (int w = 0; w < W; ++w) {
    TgWalk<KIND> walk(p, w, W);
    TgUnit u;
    while (walk.next(u)) {
      const TgShape &h = p.s[u.pi];
      if (u.mt < 0 || u.mt >= h.Mt || u.nt < 0 || u.nt >= h.Nt)
        FAIL("unit of tile %d %d of %d %d", u.mt, u.nt, h.Mt, h.Nt);
      if (u.nks < 0 || u.ks0 < 0 || (u.nks > 0 && u.ks0 + u.nks > h.kend))
        FAIL("k steps %d + %d of %d", u.ks0, u.nks, h.kend);
      const Tile t(u.pi, u.mt, u.nt);
      if (u.nks > 0 || u.whole) steps[t].emplace_back(u.ks0, u.nks);
      if (u.whole) {
        if (u.ks0 != 0 || u.nks != h.kend) FAIL("a whole tile of %d + %d steps", u.ks0, u.nks);
        continue;
      }
      const int part = tg_part(w, u.ks0 > 0, CG, CG - 1);
      if (part < 0 || part >= 2 * kTgMaxCtas) FAIL("part %d", part);
      if (!used.insert(part).second) FAIL("part %d twice", part);
      parts[t].push_back({u.ks0, u.nks, part});
    }
  }
  // the tiles that exist: rows of dW that a short piece lacks have none
  for (int pi = 0; pi < (KIND == TG_GRAD ? 2 : 1); ++pi) {
    const TgShape &h = p.s[pi];
    const int rows = (h.M + p.row_step - 1) / p.row_step;
    if (p.width <= 0) continue;
    for (int mt = 0; mt < h.Mt; ++mt)
      for (int nt = 0; nt < h.Nt; ++nt) {
        auto it = steps.find(Tile(pi, mt, nt));
        if (mt >= rows) {
          if (it != steps.end()) FAIL("a tile of rows that are not there");
          continue;
        }
        if (h.kend > 0 && it == steps.end()) FAIL("tile %d %d of %d left out", mt, nt, pi);
        if (it == steps.end()) continue;
        std::map<int, int> line;
        for (auto &s : it->second)
          if (s.second > 0 && !line.emplace(s.first, s.second).second) FAIL("steps taken twice");
        int at = 0;
        for (auto &s : line) {
          if (s.first != at) FAIL("tile %d %d of %d: step %d, not %d", mt, nt, pi, s.first, at);
          at += s.second;
        }
        if (at != h.kend) FAIL("tile %d %d of %d: %d steps of %d", mt, nt, pi, at, h.kend);
      }
  }
  if (p.width <= 0 && !steps.empty()) FAIL("units of a piece that is not there");
  return "";
}

// What tg_join adds for this piece: the lists it makes, and what its threads do
// with them.
template <int CG>
std::string join_piece(const TgPlan &p, bool last, Parts &joined) {
  const int G = p.groups;
  std::vector<TgCut> cut(G + 1);
  std::vector<int> with;  // groups that have a part
  for (int w = 0; w <= G; ++w) cut[w] = tg_cut(p, w, G);
  std::vector<int> number(G + 1);
  for (int w = 0; w < G; ++w) {
    number[w] = (int)with.size();
    if (cut[w + 1].pos > cut[w].pos) with.push_back(w);
  }
  with.push_back(G);
  for (int w = 1; w < G; ++w) {
    const TgCut &c = cut[w];
    if (!tg_first_cut(p, c, cut[w - 1].pos, last)) continue;
    const TgShape &h = p.s[c.pi];
    const int end = c.pos - c.off + h.len, a = number[w] - 1;
    if (a < 0) FAIL("no group before cut %d", w);
    int b = number[w];
    while (with[b] < G && cut[with[b]].pos < end) ++b;
    for (int lane = 0; lane < p.side; ++lane) {
      const int across = h.Nt / p.side, panel = c.tile + h.dealt;
      const int mt = panel / across, nt = (panel - mt * across) * p.side + lane;
      auto &list = joined[Tile(c.pi, mt, nt)];
      if (!list.empty()) FAIL("tile %d %d of %d joined twice", mt, nt, c.pi);
      for (int n = a; n < b; ++n)
        list.push_back({0, 0, tg_part(with[n] * p.side + lane, with[n] >= w, CG, CG - 1)});
      // the first output row that is written, and whether it is in the piece
      if (c.pi == 0 && mt * p.row_step >= p.width) FAIL("a join of rows that are not there");
    }
  }
  return "";
}

std::string same_parts(const Parts &stored, const Parts &joined, int pi) {
  for (auto &t : joined)
    if (std::get<0>(t.first) == pi && !stored.count(t.first)) FAIL("joined, but not cut");
  for (auto &t : stored) {
    if (std::get<0>(t.first) != pi) continue;
    auto it = joined.find(t.first);
    if (it == joined.end()) FAIL("cut, but not joined");
    std::map<int, int> line;  // in the order of k
    for (auto &s : t.second) line[s.k0] = s.part;
    if (line.size() != it->second.size())
      FAIL("%zu parts stored, %zu joined", line.size(), it->second.size());
    size_t i = 0;
    for (auto &s : line)
      if (it->second[i++].part != s.second) FAIL("parts out of order");
  }
  return "";
}

template <int CG, int NT>
std::string gradients(const TgSizes &S, int count, int W, bool rows_counted) {
  const int host_np = S.blocked ? tg_pieces(S.M, S.N, S.cap_boxes).np : 1;
  const TgPieces dev = tg_pieces(count, S.N, S.cap_boxes);
  const int np = S.blocked ? dev.np : 1;
  if (np > host_np) FAIL("%d pieces, %d queued", np, host_np);
  std::set<int> look;
  for (int k : {0, 1, 2, np / 2, np - 2, np - 1, np, np + 1, host_np / 2, host_np - 2, host_np - 1})
    if (k >= 0 && k < host_np) look.insert(k);
  int covered = 0;
  Parts dx_first;
  bool dx_seen = false;
  for (int k : look) {
    const TgPlan p = tg_plan<CG, TG_GRAD, NT>(S, k, count, W);
    const bool there = k < np;
    if (!there && (p.width != 0 || p.col0 != S.N))
      FAIL("piece %d of %d: column %d, width %d", k, np, p.col0, p.width);
    if (there) {
      if (p.col0 < 0 || p.width <= 0 || p.col0 > S.N - p.width)
        FAIL("piece %d of %d: column %d, width %d", k, np, p.col0, p.width);
      if (k == np - 1 && p.col0 + p.width != S.N) FAIL("the last piece ends at %d", p.col0 + p.width);
      if (S.blocked && k < np - 1 && p.width != dev.tp * 256) FAIL("width %d", p.width);
      if (S.blocked && p.col0 != k * (long long)dev.tp * 256) FAIL("column %d", p.col0);
      covered += p.width;
    }
    Parts stored, joined;
    std::string e = walk_piece<CG, TG_GRAD, NT>(p, W, stored);
    if (!e.empty()) return e;
    const bool last = k == host_np - 1;
    if (NT == 256) {
      e = join_piece<CG>(p, last, joined);
      if (!e.empty()) return e;
    }
    if (!there) stored.clear();
    e = same_parts(stored, joined, 0);
    if (!e.empty()) return "dW: " + e;
    if (there) {  // dX's parts are the same ones in every piece
      Parts dx;
      for (auto &t : stored)
        if (std::get<0>(t.first) == 1) dx.insert(t);
      for (auto &t : dx)
        if (dx_seen) {
          auto it = dx_first.find(t.first);
          if (it == dx_first.end() || it->second.size() != t.second.size())
            FAIL("dX is cut otherwise in piece %d", k);
          for (size_t i = 0; i < t.second.size(); ++i)
            if (it->second[i].part != t.second[i].part || it->second[i].k0 != t.second[i].k0)
              FAIL("dX's parts move in piece %d", k);
        }
      if (dx_seen && dx.size() != dx_first.size()) FAIL("dX's cut tiles differ in piece %d", k);
      dx_first = dx, dx_seen = true;
    }
    if (last) {
      e = same_parts(dx_first, joined, 1);
      if (!e.empty()) return "dX: " + e;
    } else {
      for (auto &t : joined)
        if (std::get<0>(t.first) == 1) FAIL("dX joined before the last piece");
    }
    if (!rows_counted && there) {  // the host's question whether to join at all
      bool any = false;
      for (int x = 1; x < p.groups; ++x) any = any || tg_cut(p, x, p.groups).off != 0;
      if (!stored.empty() && !any) FAIL("cut tiles, but no join");
    }
    if (host_np > 1)  // dX's sums between pieces
      if ((size_t)(p.s[1].Mt * CG) * p.s[1].Nt > tg_tiles(S.M, S.K)) FAIL("sums of dX do not fit");
  }
  if ((int)look.size() == host_np && covered != S.N) FAIL("%d columns of %d", covered, S.N);
  return "";
}

// 128 x 128 tiles: one piece of rows that the host knows, while all tiles run at once.
std::string small_gradients(const TgSizes &S) {
  if (S.blocked && tg_pieces(S.M, S.N, S.cap_boxes).np > 1) return "";
  const TgPlan p = tg_plan<1, TG_GRAD, 128>(S, 0, S.M, kTgMaxCtas);
  const int64_t tiles = (int64_t)p.s[0].tiles + p.s[1].tiles;
  if (tiles > kTgMaxCtas) return "";
  const std::string e = gradients<1, 128>(S, S.M, kTgMaxCtas, false);
  return e.empty() ? gradients<1, 128>(S, S.M, (int)tiles, false) : e;
}

template <int CG, int KIND, int NT>
std::string rows_product(const TgSizes &S, int count, int W) {
  const int host_np = KIND == TG_PROB ? tg_pieces(S.M, S.N, S.cap_boxes).np : 1;
  const int np = KIND == TG_PROB ? tg_pieces(count, S.N, S.cap_boxes).np : 1;
  std::set<int> look;
  for (int k : {0, 1, np - 1, np, host_np - 1})
    if (k >= 0 && k < host_np) look.insert(k);
  for (int k : look) {
    const TgPlan p = tg_plan<CG, KIND, NT>(S, k, count, W);
    if (k >= np ? p.width != 0 || p.col0 != S.N
                : p.col0 < 0 || p.width <= 0 || p.col0 > S.N - p.width)
      FAIL("piece %d of %d: column %d, width %d", k, np, p.col0, p.width);
    Parts parts;
    std::string e = walk_piece<CG, KIND, NT>(p, W, parts);
    if (!e.empty()) return e;
    if (!parts.empty()) FAIL("a product with tokens as rows is cut");
    if (KIND == TG_PROB && k < np &&
        (int64_t)p.s[0].Nt * (NT / 64) * p.pc.n_tok64 > (int64_t)S.cap_boxes)
      FAIL("%d x %d boxes of %u", p.s[0].Nt * (NT / 64), p.pc.n_tok64, S.cap_boxes);
    if (KIND == TG_PROB && p.s[0].Mt * 2 * CG > p.pc.n_tok64 && count > 0) FAIL("rows of boxes");
  }
  return "";
}

char result[512];
const char *say(const std::string &e) {
  std::snprintf(result, sizeof(result), "%s", e.c_str());
  return result;
}

}  // namespace

extern "C" {

// The vocabulary loss's gradients of M rows, `count` of them with a target (0 cap:
// the workspace's own room for boxes).
const char *check_vocab_gradients(int cg, int M, int V, int d, int count, int workers, int cap) {
  TgSizes S = {};
  S.M = M, S.N = V, S.K = d, S.blocked = 1;
  S.cap_boxes = cap > 0 ? (uint32_t)cap : (uint32_t)vocab_grad_layout(M, V, d).cap_boxes;
  const bool counted = count != M;
  std::string e = cg == 1 ? gradients<1, 256>(S, count, workers, counted)
                          : gradients<2, 256>(S, count, workers, counted);
  if (e.empty() && !counted) e = small_gradients(S);
  if (!e.empty()) return say("gradients: " + e);
  e = cg == 1 ? rows_product<1, TG_PROB, 256>(S, count, workers)
              : rows_product<2, TG_PROB, 256>(S, count, workers);
  if (e.empty() && cg == 1) e = rows_product<1, TG_PROB, 128>(S, count, workers);
  if (!e.empty()) return say("probabilities: " + e);
  e = cg == 1 ? rows_product<1, TG_LSE, 256>(S, count, workers)
              : rows_product<2, TG_LSE, 256>(S, count, workers);
  return say(e.empty() ? e : "loss: " + e);
}

// The gradients of the projections: M tokens, A [M][N] (in boxes or not), d features.
const char *check_projection_gradients(int cg, int M, int N, int d, int blocked, int workers) {
  TgSizes S = {};
  S.M = M, S.N = N, S.K = d, S.blocked = blocked;
  S.cap_boxes = blocked ? (uint32_t)project_grad_layout(M, N).cap_boxes : 0;
  std::string e = cg == 1 ? gradients<1, 256>(S, M, workers, false)
                          : gradients<2, 256>(S, M, workers, false);
  if (e.empty()) e = small_gradients(S);
  if (e.empty() && blocked)
    e = cg == 1 ? rows_product<1, TG_SILU, 256>(S, M, workers)
                : rows_product<2, TG_SILU, 256>(S, M, workers);
  return say(e);
}

int vocab_boxes(int M, int V) { return (int)tg_boxes(M, V); }

}  // extern "C"
