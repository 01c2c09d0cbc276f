// What the tile kernels of microscaled products share: one workgroup per
// [rows] x [tokens] tile of the result, 32 x 32 matrix instructions, K split
// over wavefronts (KW shares) and over workgroups.
//
// A tile is kRowWaves wavefronts along the rows (32 RT each) times TW along the
// tokens (32 NT each); each of the KW shares of K has such a set of them.
#pragma once

#include "mx_device.hpp"

namespace aqlm {

constexpr int kRowWaves = 4;

struct TileArgs {
  const uint8_t *codes;    // W
  const uint8_t *scales;
  const void *x;           // activations: halves, or codes
  const uint8_t *xscales;  // and their scales
  uint16_t *y;
  float4_t *part;          // [splits][tiles][RT * NT * 4][64 kRowWaves TW], or null
  int rows, cols, batch;   // of W and x (the result is [batch][rows])
  int row_tiles, tok_tiles, splits, groups_per_split;
};

// Workgroup -> job. Workgroups go round the 8 XCDs in turn, each with an L2 of
// its own: give every XCD one run of consecutive jobs.
__device__ __forceinline__ int xcd_job(int b, int n) {
  const int per = n >> 3, rest = n & 7, xcd = b & 7, i = b >> 3;
  return xcd * per + min(xcd, rest) + i;
}

// Tile -> place. Tiles go through the rows in bands of eight tiles of tokens,
// so that the workgroups at work on an XCD (4 x 8 tiles of its 32 CUs) share
// both rows of W and steps of x. (Uniform, but divisions run on the vector
// unit: the results go back to scalar registers.)
struct TilePlace {
  int row_tile, tok_tile;
};
__device__ __forceinline__ TilePlace tile_place(int tile, int row_tiles, int tok_tiles) {
  const int band = __builtin_amdgcn_readfirstlane(tile / (8 * row_tiles));
  const int width = min(8, tok_tiles - 8 * band), in_band = tile - 8 * band * row_tiles;
  const int row_tile = __builtin_amdgcn_readfirstlane(in_band / width);
  return {row_tile, 8 * band + in_band - row_tile * width};
}

// The scale bytes of a tile's ROWS rows for GROUPS groups of 16 blocks in LDS,
// [row][16 GROUPS], 16-byte chunk g of row r at a place that spreads the rows
// over the banks. Read from memory by each lane for its own row they cost a
// 128-byte line for every 16 bytes, which bounded the tile kernels; this way
// neighbouring lanes read a row's bytes at once. THREADS threads load them into
// registers early (load) and write them when the ones before are done with
// (store).
// Past the last row they are the last one's, past the last block 127: the codes
// there are zeros, but a NaN of another row would still show.
template <int ROWS, int THREADS, int GROUPS> struct ScaleStage {
  static constexpr int kAll = ROWS * GROUPS, kChunks = (kAll + THREADS - 1) / THREADS;
  static constexpr int kBytes = kAll * 16;
  Rsrc rs;
  int nb, rows, blk;  // blocks of a row; rows there are
  uint4 v[kChunks];
  uint32_t extra[kChunks];

  // (row0, a tile's first, is a multiple of 32: its scales begin with a whole word)
  __device__ __forceinline__ ScaleStage(const uint8_t *scales, int64_t row0, int rows_, int nb_)
      : nb(nb_), rows(rows_), blk(0) {
    rs = make_rsrc(scales + row0 * nb, (uint32_t)rows * nb);
  }
  __device__ __forceinline__ uint32_t at(int id) const {  // of chunk id's first byte
    return (uint32_t)min(id / GROUPS, rows - 1) * nb + (uint32_t)(blk + 16 * (id % GROUPS));
  }
  static __device__ __forceinline__ uint32_t place(int r, int g) {
    return (uint32_t)r * (16 * GROUPS) + (uint32_t)((g ^ ((r * GROUPS >> 4) & (GROUPS - 1))) << 4);
  }
  // blocks first .. first + 16 GROUPS - 1
  __device__ __forceinline__ void load(int first, int tid) {
    blk = first;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int id = tid + i * THREADS;
      const uint32_t to = at(id) & ~3u;
      const bool in = blk + 16 * (id % GROUPS) < nb && (kAll % THREADS == 0 || id < kAll);
      v[i] = buf_load16(rs, in ? to : kMxOOB);
      if ((nb & 3) != 0) extra[i] = buf_load4(rs, in ? to + 16 : kMxOOB);
    }
  }
  __device__ __forceinline__ void store(uint8_t *lds, int tid) {
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int id = tid + i * THREADS, r = id / GROUPS, g = id % GROUPS;
      if (kAll % THREADS != 0 && id >= kAll) break;
      const int left = nb - (blk + 16 * g);  // blocks from the chunk's first on
      uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
      if ((nb & 3) != 0) {  // the bytes lie across words
        const uint32_t from = at(id), by = from & 3u;
        uint32_t d[5] = {w[0], w[1], w[2], w[3], extra[i]};
        // A word that ends past the array reads zero; its bytes that exist are
        // read one by one (the last row's end alone).
        const uint32_t end = (uint32_t)rows * nb, word = end & ~3u, to = from & ~3u;
        if (word != end && left > 0 && to + 20 > word) {
          uint32_t tail = buf_load_u8(rs, word);
          if ((end & 3u) > 1) tail |= buf_load_u8(rs, word + 1) << 8;
          if ((end & 3u) > 2) tail |= buf_load_u8(rs, word + 2) << 16;
#pragma unroll
          for (int u = 0; u < 5; ++u) d[u] = to + 4 * u == word ? tail : d[u];
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) w[u] = __builtin_amdgcn_alignbyte(d[u + 1], d[u], by);
      }
      if (left < 16) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int keep = left - 4 * u;  // bytes of the word that are blocks
          const uint32_t m = keep <= 0 ? 0u : keep >= 4 ? ~0u : 0xFFFFFFFFu >> (32 - 8 * keep);
          w[u] = (w[u] & m) | (0x7F7F7F7Fu & ~m);
        }
      }
      *reinterpret_cast<uint4 *>(lds + place(r, g)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  // the 16 bytes of group g of row r
  static __device__ __forceinline__ uint4 read(const uint8_t *lds, int r, int g) {
    return *reinterpret_cast<const uint4 *>(lds + place(r, g));
  }
};

// Registers 4 q .. 4 q + 3 of a 32 x 32 tile.
__device__ __forceinline__ float4_t quarter(const float16_t &v, int q) {
  return float4_t{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
}

// LDS bytes of one of the four arrays through which the shares' sums pass.
template <int RT, int NT, int TW> constexpr int tile_sums_bytes() { return RT * NT * TW * kRowWaves * 1024; }

// Adds the sums of K's shares, in order, to those of share 0: a quarter of the
// registers through each array. True where the wavefront is done (it is not of
// share 0).
template <int RT, int NT, int TW, int KW>
__device__ __forceinline__ bool add_shares(float16_t (&acc)[RT][NT], int kw, int wave, int lane,
                                           uint8_t *a0, uint8_t *a1, uint8_t *a2, uint8_t *a3) {
  if constexpr (KW > 1) {
    auto slot = [&](uint8_t *a, int i, int j) __attribute__((always_inline)) {
      return reinterpret_cast<float4_t *>(a + (((i * NT + j) * kRowWaves * TW + wave) * 64 + lane) * 16);
    };
#pragma unroll 1
    for (int s = 1; s < KW; ++s) {
      __syncthreads();
      if (kw == s) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j)
              *slot(q == 0 ? a0 : q == 1 ? a1 : q == 2 ? a2 : a3, i, j) = quarter(acc[i][j], q);
      }
      __syncthreads();
      if (kw == 0) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              const float4_t v = *slot(q == 0 ? a0 : q == 1 ? a1 : q == 2 ? a2 : a3, i, j);
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[i][j][4 * q + e] += v[e];
            }
      }
    }
    return kw != 0;
  }
  return false;
}

// The tile's results: to the workspace as the registers lie where K is split
// over workgroups, else rounded into y. Register 4 q + e of a 32 x 32 tile is
// row 8 q + 4 (lane / 32) + e, token lane % 32, so a lane's values are four rows
// apart from the next lane's token; they pass through LDS (kStoreBytes of it a
// wavefront, 32 tokens at a time), from where eight lanes store the 128 bytes of
// 64 rows (four the 64 of 32) of a token: 8-byte stores from the registers took
// 15 us of 76 with 2048 x 11008 results. The caller's barrier stands between
// the last other use of that LDS and this.
template <int RT> constexpr int kStoreBytes = RT * 2048;

template <MxType T, int RT, int NT, int TW>
__device__ __forceinline__ void store_tile(const TileArgs &A, const float16_t (&acc)[RT][NT], int job,
                                           const TilePlace &at, int wave, int lane, uint8_t *lds) {
  constexpr int kThreads = 64 * kRowWaves * TW;
  const int rw = wave / TW, tw = wave % TW;
  const int row0 = (at.row_tile * kRowWaves + rw) * 32 * RT, tok0 = (at.tok_tile * TW + tw) * 32 * NT;
  if (A.splits > 1) {
    float4_t *p = A.part + (int64_t)job * (RT * NT * 4 * kThreads) + wave * 64 + lane;
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j)
        if (tok0 + 32 * j + (lane & 31) < A.batch) {
#pragma unroll
          for (int q = 0; q < 4; ++q) p[((i * NT + j) * 4 + q) * kThreads] = quarter(acc[i][j], q);
        }
    return;
  }
  if ((A.rows & 7) == 0) {
    constexpr int kChunks = 4 * RT;  // of 16 bytes, eight rows, for a token
    uint8_t *const mine = lds + wave * kStoreBytes<RT>;
    const int t = lane & 31;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int c = (4 * i + q) ^ (t & (kChunks - 1));
          *reinterpret_cast<uint2 *>(mine + (t * kChunks + c) * 16 + 8 * (lane >> 5)) =
              make_uint2(f2t<T>(acc[i][j][4 * q]) | (f2t<T>(acc[i][j][4 * q + 1]) << 16),
                         f2t<T>(acc[i][j][4 * q + 2]) | (f2t<T>(acc[i][j][4 * q + 3]) << 16));
        }
#pragma unroll
      for (int k = 0; k < kChunks / 2; ++k) {
        const int id = 64 * k + lane, tt = id / kChunks, c = id % kChunks;
        const uint4 v = *reinterpret_cast<const uint4 *>(mine + (tt * kChunks + (c ^ (tt & (kChunks - 1)))) * 16);
        const int tok = tok0 + 32 * j + tt, row = row0 + 8 * c;
        if (tok < A.batch && row < A.rows)
          *reinterpret_cast<uint4 *>(A.y + (int64_t)tok * A.rows + row) = v;
      }
    }
    return;
  }
  const bool packed = (A.rows & 3) == 0;
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int tok = tok0 + 32 * j + (lane & 31);
    if (tok >= A.batch) continue;
    uint16_t *row = A.y + (int64_t)tok * A.rows;
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        store4<T>(row, row0 + 32 * i + 8 * q + 4 * (lane >> 5), A.rows, quarter(acc[i][j], q), packed);
  }
}

// Sums of the split parts, in order of the split, rounded and stored.
template <MxType T, int RT, int NT, int TW>
__global__ __launch_bounds__(64 * kRowWaves * TW) void mx_tile_sum_kernel(const TileArgs A) {
  constexpr int kThreads = 64 * kRowWaves * TW;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int tiles = A.row_tiles * A.tok_tiles;
  const int slot = (int)blockIdx.x % (RT * NT * 4), tile = (int)blockIdx.x / (RT * NT * 4);
  const float4_t *p = A.part + ((int64_t)tile * (RT * NT * 4) + slot) * kThreads + tid;
  const int64_t stride = (int64_t)tiles * (RT * NT * 4) * kThreads;
  const TilePlace at = tile_place(tile, A.row_tiles, A.tok_tiles);
  const int q = slot & 3, j = (slot >> 2) % NT, i = (slot >> 2) / NT;
  const int tok = (at.tok_tile * TW + wave % TW) * 32 * NT + 32 * j + (lane & 31);
  const int row = (at.row_tile * kRowWaves + wave / TW) * 32 * RT + 32 * i + 8 * q + 4 * (lane >> 5);
  if (tok >= A.batch) return;
  float4_t v = p[0];
  for (int s = 1; s < A.splits; s += 4) {  // four loads under way
    float4_t u[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) u[k] = p[min(s + k, A.splits - 1) * stride];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (s + k < A.splits) v += u[k];
  }
  store4<T>(A.y + (int64_t)tok * A.rows, row, A.rows, v, (A.rows & 3) == 0);
}

// Tile of a product and the workgroups K is split over: the choice with the
// shortest modelled time. The grid runs in rounds of up to 256 workgroups, one
// per CU, and a group of K takes a + b * (workgroups of the round / 256) us for
// each share; 2.7 us pass around that; a split writes and reads its sums at about
// 4 TB/s and launches a second kernel.
struct TileShape {
  int rt, nt, tw, kw;
  double a, b;
};

struct TilePlan {
  TileShape shape;
  int splits, groups_per_split;
  int64_t row_tiles, tok_tiles;
  double us;  // modelled
  int64_t ws_bytes() const {
    if (splits == 1) return 0;
    return row_tiles * tok_tiles * splits * (int64_t)(shape.rt * shape.nt * shape.tw * kRowWaves) * 4096;
  }
};

// `most`: the largest number of splits (1: no workspace).
template <int N>
TilePlan plan_tiles(const TileShape (&shapes)[N], int64_t rows, int64_t batch, int64_t groups,
                    int most = 8) {
  TilePlan best{};
  for (const TileShape &c : shapes) {
    TilePlan p{};
    p.shape = c;
    p.row_tiles = (rows + 32 * kRowWaves * c.rt - 1) / (32 * kRowWaves * c.rt);
    p.tok_tiles = (batch + 32 * c.nt * c.tw - 1) / (32 * c.nt * c.tw);
    const int64_t tiles = p.row_tiles * p.tok_tiles;
    for (int s = 1; s <= most; ++s) {
      p.groups_per_split = (int)((groups + s - 1) / s);
      p.splits = (int)((groups + p.groups_per_split - 1) / p.groups_per_split);
      if (p.splits != s || (s > 1 && tiles * s > 256)) break;
      const double whole = (double)(tiles * s / 256), rest = (double)(tiles * s % 256) / 256.0;
      const double group = whole * (c.a + c.b) + (rest > 0 ? c.a + c.b * rest : 0.0);
      double us = 2.7 + (double)((p.groups_per_split + c.kw - 1) / c.kw) * group;
      if (s > 1) us += 2.3 + (double)p.ws_bytes() * 2.0 / 4e6;
      p.us = us;
      if (best.splits == 0 || us < best.us) best = p;
    }
  }
  return best;
}

inline TileArgs tile_args(const TilePlan &p, const MxDesc &W, const void *x, const uint8_t *xscales,
                          int64_t batch, void *y, void *ws) {
  return {W.codes, W.scales, x, xscales, static_cast<uint16_t *>(y), static_cast<float4_t *>(ws),
          (int)W.rows, (int)W.cols, (int)batch, (int)p.row_tiles, (int)p.tok_tiles, p.splits,
          p.groups_per_split};
}

}  // namespace aqlm
