// tg_plan.h -- the schedule of the training operators' products (tc_tgemm.cuh):
// pieces of the column axis, tiles, their cuts along k and the order in which a
// worker takes them.  Every warp of a kernel works it out by itself from the
// sizes and the device's row count; the host uses it to choose launches, and
// tests/test_train_schedule.py walks it on the CPU.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace fmca {
namespace {

enum : int { TG_LSE = 0, TG_PROB = 1, TG_SILU = 2, TG_GRAD = 3 };

// What the schedule depends on beside the row count and the workers.
struct TgSizes {
  int M, N, K;         // NT: rows, columns, depth; TG_GRAD: tokens, columns of A (V), features
  int blocked;         // TG_GRAD: A lies in boxes
  uint32_t cap_boxes;  // room for boxes
};

// Pieces of the column axis: as many 256-column tiles a piece as the boxes of
// all tokens fit the buffer, the pieces equal in length.
struct TgPieces {
  int n_tok64, tiles, tp, np;
};
__host__ __device__ inline TgPieces tg_pieces(int count, int V, uint32_t cap_boxes) {
  TgPieces r;
  r.n_tok64 = (count > 0 ? (int)(((uint32_t)count + 255) / 256) : 1) * 4;
  r.tiles = (int)(((uint32_t)V + 255) / 256);
  uint32_t tp = cap_boxes / (4 * (uint32_t)r.n_tok64);
  if (tp < 1) tp = 1;
  if (tp > (uint32_t)r.tiles) tp = r.tiles;
  r.np = (int)(((uint32_t)r.tiles + tp - 1) / tp);
  r.tp = (int)(((uint32_t)r.tiles + r.np - 1) / (uint32_t)r.np);
  return r;
}

// One of a launch's products: rows that exist, tiles of 128 CG rows and of 256
// columns, k steps in a full piece and in this one; TG_GRAD: panels that are
// dealt out whole, panels that are cut, the length of one of those.
struct TgShape {
  int M, Mt, Nt, ks, kend, tiles, dealt, cut, len;
};
struct TgPlan {
  int count, col0, width;   // rows; first column and columns of the piece
  TgPieces pc;
  TgShape s[2];
  int base1, total;         // TG_GRAD: where problem 1's cut panels begin, and end
  bool apart;               // the panels left over are not cut: one a group
  int row_step;             // rows of a tile
  int side, groups;         // tiles of a panel, workers side by side on them
};

// A tile's epilogue beyond what the next tile's products hide, in k steps.
constexpr int kTgEpilogue = 3;
// The launch that joins the parts of cut tiles (5 us), in k steps.
constexpr int kTgJoin = 14;

template <int CG, int NT>
__host__ __device__ inline TgShape tg_shape(int M_exist, int M, int N, int K, int K_full,
                                            int side, int groups) {
  TgShape h;
  h.M = M_exist;
  h.Mt = (M + 128 * CG - 1) / (128 * CG);
  h.Nt = (N + NT - 1) / NT;
  h.ks = (K_full + 63) / 64;
  h.kend = (K + 63) / 64;
  h.tiles = h.Mt * h.Nt;
  h.dealt = h.tiles / side / groups * groups;
  h.cut = h.tiles / side - h.dealt;
  h.len = h.ks + kTgEpilogue;
  return h;
}

template <int CG, int KIND, int NT = 256>
__host__ __device__ inline TgPlan tg_plan(const TgSizes &P, int piece, int count, int workers) {
  TgPlan p;
  p.count = count;
  p.row_step = 128 * CG;
  if (KIND != TG_LSE) p.pc = tg_pieces(count, P.N, P.cap_boxes);
  p.col0 = 0;
  p.width = P.N;
  int full = P.N;
  if (KIND == TG_PROB || (KIND == TG_GRAD && P.blocked)) {
    // a piece that the row count leaves out begins behind the last column and has
    // none: the host queues the pieces of all rows, and far more narrow pieces than
    // there are wide ones times `full` would not fit 32 bits
    const bool there = piece < p.pc.np;
    full = p.pc.tp * 256;
    p.col0 = there ? piece * full : P.N;
    p.width = P.N - p.col0 < full ? P.N - p.col0 : full;
  }
  p.side = 1;
  if (KIND == TG_GRAD && NT == 256) {
    // as many tiles of a row panel side by side as leave few workers over;
    // only where one of the products is all cut
    const int Nt = (P.K + 255) / 256, rows = 128 * CG;
    if (((full + rows - 1) / rows) * Nt < workers || ((count + rows - 1) / rows) * Nt < workers)
      for (int g = 2; g <= 6; ++g)
        if (Nt % g == 0 && workers % g <= workers / 32) p.side = g;
  }
  p.groups = workers / p.side;
  if (KIND == TG_GRAD) {
    // dW [width][K], depth tokens; dX [tokens][K], depth width.  The tiles and
    // their cuts are those of a full piece in every piece, so that the sums of
    // dX go on from piece to piece; the last one leaves some without work.
    p.s[0] = tg_shape<CG, NT>(p.width, full, P.K, count, count, p.side, p.groups);
    p.s[1] = tg_shape<CG, NT>(count, count, P.K, p.width, full, p.side, p.groups);
    // fewer cut panels than workers, 2^22 steps each at most: 31 bits hold it
    p.base1 = p.s[0].cut * p.s[0].len;
    p.total = p.base1 + p.s[1].cut * p.s[1].len;
    // no cuts where they would save less than joining the parts takes
    const int len0 = p.s[0].cut ? p.s[0].len : 0, len1 = p.s[1].cut ? p.s[1].len : 0;
    p.apart = NT < 256 || (p.s[0].cut + p.s[1].cut <= p.groups &&
                           (len0 > len1 ? len0 : len1) <= p.total / p.groups + kTgJoin);
  } else {
    p.s[0] = tg_shape<CG, NT>(count, p.width > 0 ? count : 0, p.width, P.K, P.K, 1, workers);
    p.s[1] = p.s[0];
    p.base1 = p.total = 0;
    p.apart = false;
  }
  return p;
}

// TG_GRAD's work: a panel is up to 6 tiles side by side (the same rows of A),
// one for each worker of a group, which read A together at the same time.  Of
// either problem as many panels as make whole rounds of all groups are dealt
// out, neighbours at the same time.  What is left of both is one line of k
// steps, problem 0's panels and then problem 1's, cut into equal parts, one a
// group: dealt out whole, the last panels would leave most workers idle (189
// tiles of 128 steps and 96 of 252 on 76 pairs: busy 84 % of the time).  The
// tiles of a panel that a cut goes through are summed from their parts by a
// second kernel; a part keeps 8 k steps at least, and panels of less than 16
// are not cut, nor any where that kernel costs more than the cuts save.  Without
// panels (each worker on a tile of its own, cut at its own place) A came from
// DRAM once for every tile beside another: the loss's gradients of 2048 x 50001 x
// 512 take 242 us, without panels 267.  Where group w's part of the line begins:
struct TgCut {
  int pi, tile, off;  // the panel among the cut ones; k steps of it before the cut
  int pos;
};
__host__ __device__ inline TgCut tg_cut(const TgPlan &p, int w, int W) {
  TgCut c;
  if (p.apart) {
    const int n0 = p.s[0].cut, n = n0 + p.s[1].cut;
    if (w > n) w = n;
    c.pi = w >= n0 ? 1 : 0;
    c.tile = c.pi ? w - n0 : w;
    c.off = 0;
    c.pos = c.pi ? p.base1 + c.tile * p.s[1].len : w * p.s[0].len;
    return c;
  }
  const int b = w <= 0 ? 0 : w >= W ? p.total : w * (p.total / W) + w * (p.total % W) / W;
  c.pi = b >= p.base1 ? 1 : 0;
  const int len = c.pi ? p.s[1].len : p.s[0].len, ks = c.pi ? p.s[1].ks : p.s[0].ks;
  const int at = c.pi ? b - p.base1 : b;
  c.tile = at / len;
  int off = at - c.tile * len;
  if (ks < 16) {
    off = 2 * off >= len ? len : 0;
  } else {
    off = (off + 4) / 8 * 8;
    if (off > ks - 8) off = len;
  }
  c.pos = (c.pi ? p.base1 : 0) + c.tile * len + off;
  if (off == len) {  // the beginning of the next panel
    ++c.tile;
    off = 0;
    if (c.pi == 0 && c.tile == p.s[0].cut) c.pi = 1, c.tile = 0;
  }
  c.off = off;
  return c;
}

struct TgUnit {
  int pi, mt, nt, ks0, nks;
  bool whole;  // the tile's whole depth
};
// A worker's units in order (every role of the kernel walks them by itself).
// The products with their tokens as rows: dealt round-robin, in blocks of 64
// row tiles (so that a block's rows and the columns at hand stay in L2), rows
// first within a block.
template <int KIND>
struct TgWalk {
  const TgPlan &p;
  int W, pi, u;  // workers (TG_GRAD: groups); next tile (panel) to be dealt
  int lane;      // worker of its group
  bool out = false;
  TgCut c;       // TG_GRAD: where the next part begins
  int end;
  __host__ __device__ TgWalk(const TgPlan &plan, int w, int workers) : p(plan) {
    start(w, workers);
  }
  // (one that is started later)
  __host__ __device__ explicit TgWalk(const TgPlan &plan) : p(plan) {}
  __host__ __device__ void start(int w, int workers) {
    W = workers;
    pi = 0;
    u = w;
    lane = 0;
    if (KIND == TG_GRAD) {
      W = p.groups;
      u = w / p.side;
      lane = w - u * p.side;
      out = u >= W;
      c = tg_cut(p, u, W);
      end = tg_cut(p, u + 1, W).pos;
    }
  }
  __host__ __device__ bool next(TgUnit &o) {
    if (KIND != TG_GRAD) {
      const TgShape &h = p.s[0];
      if (u >= h.tiles) return false;
      constexpr int kBlock = 64;
      const int per = kBlock * h.Nt, b = u / per, v = u % per;
      const int rows = h.Mt - b * kBlock < kBlock ? h.Mt - b * kBlock : kBlock;
      o.pi = 0;
      o.mt = b * kBlock + v % rows;
      o.nt = v / rows;
      o.ks0 = 0;
      o.nks = h.ks;
      o.whole = true;
      u += W;
      return true;
    }
    // a piece behind the last; a worker that belongs to no group
    if (p.width <= 0 || out) return false;
    while (true) {
      int tile;
      if (pi == 0 && u >= p.s[0].dealt) {
        u -= p.s[0].dealt;  // the rounds are whole: the group's place is the same
        pi = 1;
      }
      if (pi == 0 || u < p.s[1].dealt) {
        o.pi = pi;
        o.ks0 = 0;
        o.nks = pi ? p.s[1].kend : p.s[0].kend;
        o.whole = true;
        tile = u;
        u += W;
      } else if (c.pos < end) {
        const TgShape &h = c.pi ? p.s[1] : p.s[0];
        o.pi = c.pi;
        o.ks0 = c.off;
        tile = h.dealt + c.tile;
        int k1 = h.ks;
        if (end - c.pos < h.len - c.off) k1 = c.off + (end - c.pos);
        o.whole = c.off == 0 && k1 == h.ks;
        o.nks = (k1 < h.kend ? k1 : h.kend) - c.off;
        if (o.nks < 0) o.nks = 0;
        if (k1 < h.ks) {
          c.pos = end;
        } else {
          c.pos += h.len - c.off;
          c.off = 0;
          if (++c.tile == h.cut && c.pi == 0) c.pi = 1, c.tile = 0;
        }
      } else {
        return false;
      }
      const int across = p.s[0].Nt / p.side;  // panels of a row of tiles
      o.mt = tile / across;
      o.nt = (tile - o.mt * across) * p.side + lane;
      // rows of dW that a short last piece does not have
      if (o.pi == 0 && o.mt * p.row_step >= p.s[0].M) continue;
      return true;
    }
  }
};

// The fp32 part that a CTA keeps of a tile that was begun by another worker (its
// first) or is ended by another (its last).
__host__ __device__ inline int tg_part(int worker, bool begun, int cg, int rank) {
  return (2 * worker + (begun ? 0 : 1)) * cg + rank;
}
// Whether cut c, where a group's part of the line begins and the group before it
// began at `before`, is the first of a panel whose tiles tg_join completes:
// dW: this piece's rows; dX: complete once every piece has been.
__host__ __device__ inline bool tg_first_cut(const TgPlan &p, const TgCut &c, int before,
                                             bool last) {
  if (c.off == 0 || before > c.pos - c.off) return false;
  const int panel = c.tile + p.s[c.pi].dealt, mt = panel / (p.s[0].Nt / p.side);
  return c.pi == 0 ? mt * p.row_step < p.s[0].M : last;
}

}  // namespace
}  // namespace fmca
