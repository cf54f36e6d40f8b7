// Body of the tile kernel (nm_tile.hpp includes it, with TILE_RETURN as its return):
// the items of a workgroup.  In scope: the template arguments, a, list, list2, lds
// and `first`, from which of the XCD's workgroups on TILE_COLS deals w.lead items
// ahead of the rest.  It leaves `more`: TILE_ROWS, how many of the XCD's workgroups
// have one item more than the others.
  constexpr bool EROWS = OP == TILE_ROWS, COLS = OP == TILE_COLS, GROUPED = grouped_op(OP);
  typedef typename std::conditional<ET == TILE_I8, v4i, v4f>::type Acc;
  constexpr int NW = WM * WN;
  constexpr int TM = BM / WM / 16, TN = BN / WN / 16;   // 16 x 16 tiles of a wave
  constexpr bool MX = ET == TILE_MX;
  constexpr bool GLU = OP == TILE_GLU;
  constexpr bool BACK = OP == TILE_BACK;
  constexpr int ROWS = BM + BN;
  constexpr int DATA = ROWS * 128;
  constexpr int STAGE = DATA + (MX ? ROWS * 8 : 0);
  constexpr int NL = ROWS / 8 / NW;                     // 1 KB loads of a wave per slab
  constexpr int NLA = BM / 8 / NW;                      // of them A rows
  constexpr int NU = MX ? ROWS / 32 : 0;                // scale units per slab
  constexpr int NLT = NL + (NU + NW - 1) / NW;          // loads of a wave per slab
  constexpr int BNO = GLU ? BN / 2 : BN;                // outputs per tile
  constexpr int HB = BN / WN / 2;                       // TILE_GLU: rows per half
  constexpr int RJ = 8 * NW;                            // rows one load of every wave covers
  static_assert(BM % RJ == 0 && BN % RJ == 0, "every load of one operand");
  static_assert(!GLU || HB % RJ == 0 || RJ % (2 * HB) == 0, "a wave's load has rows of one weight");
  static_assert(tile_lds<ET, OP, BM, BN, NS>() <= 160 * 1024, "LDS");
  static_assert(!MX || !GLU || HB % 32 == 0, "whole scale units per half");

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int li = lane & 15, lq = lane >> 4;
  const int wm = wave % WM, wn = wave / WM;

  const auto walk = [&]() {
    if constexpr (GROUPED)
      return RowsWalk<BM, COLS, kRowsTable>(a, list.mt, list.nt, reinterpret_cast<int*>(lds + NS * STAGE), first);
    else
      return TileWalk<BACK>(list, list2, a.w.lead);
  }();
  if constexpr (EROWS) zero_other_rows<OUT>(a, walk.row_at);
  int more = 0;
  if constexpr (EROWS) more = walk.more;
  if (walk.count <= 0) TILE_RETURN;

  // ---- operand loads: load d fills LDS rows 8 d .. 8 d + 7, lane l row
  // 8 d + l / 8, position l % 8 = piece (l % 8) ^ (l / 8); wave w issues
  // d = w + NW j
  const int piece = (lane & 7) ^ (lane >> 3);
  // TILE_GLU with the RJ rows of a load spanning both halves: a wave's rows are all gate or all up rows
  constexpr bool SPAN = GLU && HB % RJ != 0;
  const bool wave_up = SPAN && (8 * wave / HB & 1);
  // TILE_COLS: an operand's slab is 64 rows of BM (BN) columns as they lie in memory,
  // read transposed from LDS; load d of it fills 1 KB, 16-byte position p of row t
  // with piece p ^ 2 swz(t).  A read's sixteen lanes take 32 bytes each of four rows
  // (t & 3), the next sixteen those eight rows on: all on different banks.
  auto swz = [](int t, auto width) {
    return decltype(width)::value >= 128 ? (t & 3) | (t >> 3 & 1) << 2 : (t >> 1 & 1) | (t >> 3 & 1) << 1;
  };
  // row of the tile (A: of BM, B: of BNO outputs) that load j brings this lane
  auto load_row = [&](auto jc) {
    constexpr int j = decltype(jc)::value;
    int row = 8 * wave + (lane >> 3) + RJ * j;
    if constexpr (j >= NLA) {
      row -= BM;
      if constexpr (GLU) row = row / (2 * HB) * HB + row % HB;
    }
    return row;
  };
  // pieces past the end of a row, in the last slab: an offset no resource holds
  // (TILE_BACK: rows of whole slabs)
  const int cut_a = !BACK && !COLS && (a.ka & 7) && piece >= (a.ka & 7) ? (int)0x80000000 : 0;
  const int cut_b = !BACK && !GROUPED && (a.kb & 7) && piece >= (a.kb & 7) ? (int)0x80000000 : 0;

  // the load cursor: work item, its resources, next slab
  // (TILE_COLS: rows left, ends of a row in the resources, slabs with short ones in flight)
  int ck = 0, cs, ce, cleft, cend_a, cend_b, short_slabs = 0, voff[NL];
  v4i ra, rb0, rb1, rsc[MX ? (NU + NW - 1) / NW : 1];
  // (always inlined: a call would keep the cursor, and what it refers to, in memory)
  // TILE_COLS: rows past the expert's last are past the resources' ends, zeros
  auto limit_rows = [&]() __attribute__((always_inline)) {
    const int n = min(cleft, 64);
    ra[2] = scalar(n > 0 ? (n - 1) * (int)a.lda + cend_a : 0);
    rb0[2] = scalar(n > 0 ? (n - 1) * (int)a.ldb + cend_b : 0);
  };
  auto cursor_item = [&](int k) __attribute__((always_inline)) {
    const TileItem it = walk.item(k);
    const int64_t m0 = EROWS ? (int64_t)it.row : (int64_t)it.m * BM, n0 = (int64_t)it.n * BNO;
    auto tile_rsrc = [&](const uint8_t* p, int64_t row0, int64_t ld) {
      const v4i r = make_rsrc(p + row0 * ld, 0x7fffffff);
      return v4i{scalar(r[0]), scalar(r[1]), r[2], r[3]};
    };
    const bool grad = BACK && it.batch;                 // a weight gradient
    const int64_t Mr = EROWS ? (int64_t)it.end : grad ? a.w.Mr : a.Mr, Nr = grad ? a.w.Nr : a.Nr;
    const int64_t lda = grad ? a.w.ld : a.lda, ldb = grad ? a.w.ld : a.ldb;
    const int mlast = (int)min(Mr - m0, (int64_t)BM) - 1, nlast = (int)min(Nr - n0, (int64_t)BNO) - 1;
    static_for<0, NL>([&](auto jc) {
      constexpr int j = decltype(jc)::value;
      if constexpr (COLS) {
        constexpr int W = j < NLA ? BM : BN, PC = W / 8;
        const int d = wave + NW * (j < NLA ? j : j - NLA), t = d * (64 / PC) + lane / PC;
        voff[j] = t * (int)(j < NLA ? lda : ldb) + 16 * (lane % PC ^ 2 * swz(t, ic<W>()));
      } else if constexpr (EROWS && j >= NLA) {          // blocks of 16 rows
        const int row = min(load_row(jc), nlast);
        voff[j] = (row >> 4) * (a.nslab * 2048) + (row & 15) * 128 + 16 * piece;
      } else {
        voff[j] = j < NLA ? min(load_row(jc), mlast) * (int)lda + 16 * piece
                          : min(load_row(jc), nlast) * (int)ldb + 16 * piece;
      }
    });
    ra = tile_rsrc(grad ? (it.batch > 1 ? a.w.A[1] : a.w.A[0]) : a.A, COLS ? 0 : m0, lda);
    if constexpr (EROWS)
      rb0 = tile_rsrc(a.B[0], (int64_t)it.batch * ((a.Nr + 15) / 16) + n0 / 16, (int64_t)a.nslab * 2048);
    else
      rb0 = tile_rsrc(grad ? a.w.B : wave_up ? a.B[1] : a.B[0], COLS ? 0 : n0, ldb);
    if constexpr (GLU && !SPAN) rb1 = tile_rsrc(a.B[1], n0, ldb);
    if constexpr (MX) {
      // unit u of a stage: LDS rows 32 u ..; row groups past the end repeat the last one
      static_for<0, (NU + NW - 1) / NW>([&](auto jc) {
        constexpr int j = decltype(jc)::value;
        const int u = min(wave + NW * j, NU - 1);
        const uint8_t* base = a.As;
        int64_t g32 = min(m0 / 32 + u, (a.Mr - 1) / 32);
        if (u >= BM / 32) {
          int row = 32 * u - BM;
          base = a.Bs[0];
          if constexpr (GLU) {
            if (row / HB & 1) base = a.Bs[1];
            row = row / (2 * HB) * HB + row % HB;
          }
          g32 = min((n0 + row) / 32, (a.Nr - 1) / 32);
        }
        const v4i r = make_rsrc(base + g32 * a.nslab * 256, 0);
        rsc[j] = v4i{scalar(r[0]), scalar(r[1]), scalar(a.nslab * 256), r[3]};
      });
    }
    cs = it.s0;
    ce = it.s1;
    if constexpr (COLS) {
      auto at = [&](v4i& r, const uint8_t* p) {
        const v4i q = make_rsrc(p, 0);
        r[0] = scalar(q[0]);
        r[1] = scalar(q[1]);
      };
      at(ra, a.A + it.row * a.lda + m0 * 2);
      at(rb0, a.B[0] + it.row * a.ldb + n0 * 2);
      cleft = it.end - it.row;
      cend_a = a.ka * 16 - (int)m0 * 2;
      cend_b = a.kb * 16 - (int)n0 * 2;
      limit_rows();
    }
  };
  auto issue_one = [&](auto jc, int st, int ca, int cb) {
    constexpr int j = decltype(jc)::value;
    uint8_t* sp = lds + st * STAGE;
    if constexpr (j < NL) {
      const int so = COLS ? 0 : scalar(cs * (EROWS && j >= NLA ? 2048 : 128));
      const uint32_t dst = lds_addr(sp + 1024 * (wave + NW * j));
      constexpr bool UP = GLU && !SPAN && ((RJ * j - BM) / HB & 1);
      lds_dma16(j < NLA ? ra : (UP ? rb1 : rb0), dst, voff[j] | (j < NLA ? ca : cb), so);
    } else {
      // (a wave without a unit of its own repeats the last one: no branch among the products)
      const int u = min(wave + NW * (j - NL), NU - 1);
      lds_dma4(rsc[j - NL], lds_addr(sp + DATA + 256 * u), 4 * lane, cs * 256);
    }
  };
  // part p of NP of the cursor slab's loads into stage st
  auto issue_part = [&](auto pc, auto npc, int st) {
    constexpr int P = decltype(pc)::value, NP = decltype(npc)::value;
    const int ca = BACK || COLS || cs + 1 < a.nslab ? 0 : cut_a;
    const int cb = BACK || GROUPED || cs + 1 < a.nslab ? 0 : cut_b;
    if constexpr (COLS && P == 0) short_slabs = cleft < 64 ? NS : max(short_slabs - 1, 0);
    static_for<NLT * P / NP, NLT * (P + 1) / NP>([&](auto jc) { issue_one(jc, st, ca, cb); });
  };
  // the loads of the slab after the one multiplied are in
  auto wait_loads = [&](auto lgkm) __attribute__((always_inline)) {
    constexpr int AHEAD = NLT * (NS - 2);               // loads that may be outstanding then
    static_assert(AHEAD < 64, "vmcnt");
    __builtin_amdgcn_s_waitcnt(waitcnt(AHEAD, decltype(lgkm)::value));
    if constexpr (COLS && AHEAD > 0)
      if (short_slabs) __builtin_amdgcn_s_waitcnt(waitcnt(0, 15));
  };
  // past the last work item the cursor stays on its last slab: the loads fill
  // a stage nobody reads
  auto advance = [&]() __attribute__((always_inline)) {
    if (__builtin_expect(cs + 1 < ce, 1)) {
      ++cs;
      if constexpr (COLS) {
        auto next_slab = [](v4i& r, int64_t bytes) __attribute__((always_inline)) {
          const uint64_t p = ((uint64_t)(uint32_t)r[1] << 32 | (uint32_t)r[0]) + bytes;
          r[0] = (int)p;
          r[1] = (int)(p >> 32);
        };
        next_slab(ra, a.lda * 64);
        next_slab(rb0, a.ldb * 64);
        cleft -= 64;
        limit_rows();
      }
    } else if (ck + 1 < walk.count) {
      asm volatile("" ::: "memory");                    // a branch, not selects around it
      cursor_item(++ck);
    }
  };

  Acc acc[TN][TM];
  auto clear = [&]() {
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int j = 0; j < TM; ++j) acc[i][j] = Acc{0, 0, 0, 0};
  };
  clear();

  // fragment addresses: row li of a 16-row tile, piece 4 kk + lq
  const int arow = (wm * TM * 16 + li) * 128;
  const int brow = (BM + wn * TN * 16 + li) * 128;
  // (TILE_COLS: its rows' first half and second)
  const int pos0 = COLS ? 0 : 16 * (lq ^ (li & 7)), pos1 = COLS ? 1 : 16 * ((4 + lq) ^ (li & 7));
  // TILE_COLS: of column tile X rows 8 lq + 4 h .. + 3; lane li brings row li / 4's
  // columns 4 (li % 4) .. and takes column li of all four
  int acol[COLS ? TM : 1], bcol[COLS ? TN : 1];
  if constexpr (COLS) {
    const int t = 8 * lq + (li >> 2);
#pragma unroll
    for (int x = 0; x < TM; ++x) acol[x] = t * (2 * BM) + (wm * TM + x ^ swz(t, ic<BM>())) * 32 + 8 * (li & 3);
#pragma unroll
    for (int x = 0; x < TN; ++x)
      bcol[x] = BM * 128 + t * (2 * BN) + (wn * TN + x ^ swz(t, ic<BN>())) * 32 + 8 * (li & 3);
  }
  struct Frag {
    v4i a[TM], b[TN];
  };
  constexpr int NF = TM + TN;
  auto read_one = [&](Frag& f, auto xc, int st, int pos) {
    constexpr int X = decltype(xc)::value;
    if constexpr (COLS) {
      constexpr bool A = X < TM;
      constexpr int pitch = 2 * (A ? BM : BN);
      const uint8_t* sp = lds + st * STAGE + (A ? acol[A ? X : 0] : bcol[A ? 0 : X - TM]) + pos * (32 * pitch);
      const v2i lo = lds_tr16(sp), hi = lds_tr16(sp + 4 * pitch);
      (A ? f.a[A ? X : 0] : f.b[A ? 0 : X - TM]) = v4i{lo[0], lo[1], hi[0], hi[1]};
      return;
    }
    const uint8_t* sp = lds + st * STAGE + pos;
    if constexpr (X < TM)
      f.a[X] = *reinterpret_cast<const v4i*>(sp + arow + X * 2048);
    else
      f.b[X - TM] = *reinterpret_cast<const v4i*>(sp + brow + (X - TM) * 2048);
  };
  struct Scales {
    int a[MX ? TM / 2 : 1], b[MX ? TN / 2 : 1];
  };
  auto read_scales = [&](Scales& f, int st) {
    if constexpr (MX) {
      const uint8_t* sp = lds + st * STAGE + DATA + 4 * lane;
#pragma unroll
      for (int j = 0; j < TM / 2; ++j) f.a[j] = *reinterpret_cast<const int*>(sp + (wm * TM / 2 + j) * 256);
#pragma unroll
      for (int i = 0; i < TN / 2; ++i) f.b[i] = *reinterpret_cast<const int*>(sp + (BM / 32 + wn * TN / 2 + i) * 256);
    }
  };
  auto mul_row = [&](auto ic_, auto kc, const Frag& f, const Scales& c) {
    constexpr int i = decltype(ic_)::value, kk = decltype(kc)::value;
    // back and forth: one operand stays at the turn too (what changes at the
    // matrix cores' inputs costs power: 2-4% of the forward products)
#pragma unroll
    for (int q = 0; q < TM; ++q) {
      const int j = i & 1 ? TM - 1 - q : q;
      if constexpr (MX)
        acc[i][j] = mfma_mx(f.b[i], f.a[j], acc[i][j], c.b[i / 2], 2 * (i & 1) + kk, c.a[j / 2], 2 * (j & 1) + kk);
      else if constexpr (ET == TILE_I8)
        acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(f.b[i], f.a[j], acc[i][j], 0, 0, 0);
      else
        acc[i][j] = mfma_16<ET>(f.b[i], f.a[j], acc[i][j]);
    }
  };

  // Slab s: its second half's fragments are read between the products of the
  // first half; then, with slab s + 1 landed and every wave done reading slab
  // s, the first fragments of slab s + 1 are read and the loads of slab
  // s + NS go out into s's stage between the products of the second half.
  cursor_item(0);
  static_for<0, NS - 1>([&](auto k) {
    issue_part(ic<0>(), ic<1>(), decltype(k)::value);
    advance();
  });
  wait_loads(ic<15>());
  barrier_nofence();
  issue_part(ic<0>(), ic<1>(), NS - 1);
  advance();
  Frag f0, f1;
  Scales c0, c1;
  static_for<0, NF>([&](auto x) { read_one(f0, x, 0, pos0); });
  read_scales(c0, 0);
  int st = 0;
  for (int k = 0; k < walk.count; ++k) {
    const TileItem it = walk.item(k);
    const int64_t m0 = (EROWS ? (int64_t)it.row : (int64_t)it.m * BM) + wm * TM * 16;
    const int64_t n0 = (int64_t)it.n * BNO + wn * (BNO / WN);
    v4i kept = {0, 0, 0, 0};
    if constexpr (COLS) {
      if (m0 < a.Mr && n0 < a.Nr)
        kept = *reinterpret_cast<const v4i*>(
            a.mask + ((it.batch * ((a.Mr + 127) / 128) + (m0 >> 7)) * a.ldm + (n0 >> 6)) * 1024 + 16 * lane);
    }
    for (int s = it.s0; s < it.s1; ++s) {
      static_for<0, TN>([&](auto i) {
        constexpr int I = decltype(i)::value;
        static_for<NF * I / TN, NF * (I + 1) / TN>([&](auto x) { read_one(f1, x, st, pos1); });
        __builtin_amdgcn_sched_barrier(0);
        mul_row(i, ic<0>(), f0, c0);
        __builtin_amdgcn_sched_barrier(0);
      });
      wait_loads(ic<0>());
      barrier_nofence();
      const int nx = st + 1 == NS ? 0 : st + 1;
      read_scales(c1, nx);
      static_for<0, TN>([&](auto i) {
        constexpr int I = decltype(i)::value;
        static_for<NF * I / TN, NF * (I + 1) / TN>([&](auto x) { read_one(f0, x, nx, pos0); });
        issue_part(i, ic<TN>(), st);
        __builtin_amdgcn_sched_barrier(0);
        mul_row(i, ic<1>(), f1, c0);
        __builtin_amdgcn_sched_barrier(0);
      });
      // the products stay above the cursor's branch (sunk below it they would
      // keep every fragment of the slab alive)
#pragma unroll
      for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j) asm volatile("" : "+v"(acc[i][j]));
      advance();
      c0 = c1;
      st = nx;
    }
    if constexpr (COLS) {
      tile_cols<OUT>(a, it, m0, n0, kept, acc);
    } else if constexpr (EROWS) {
      rows_epilogue<OUT, TM, TN>(a, it, m0, n0, acc);
    } else {
      tile_epilogue<OP, OUT, TM, TN>(a, it, m0, n0, acc);
    }
    clear();
  }
  __builtin_amdgcn_s_waitcnt(waitcnt(0, 15));           // nothing lands in LDS after this
