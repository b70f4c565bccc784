// The body of the attention kernels (sv_attend_kernel.h says how it works): statements of a
// function that has
//   the template arguments D, F8, MT, PG16;
//   constexpr bool OWN: of request r only the positions from a.first[r] on (below 0: the
//     request is left alone), always into partial results;
//   a (AttendArgs); block, blocks: this workgroup and how many there are;
//   sm (Attend<D, F8, MT, PG16>::Smem).
// Included, not called: as a function inlined into sv_cache_attend's kernel hipcc gave it 128 ..
// 139 accumulation registers at 256 dims instead of 72 .. 82, which cost 1 .. 4 % (128 x 1
// row, 16 heads over 4, ctx 4096: 262 -> 273 us), and rounded some results otherwise than before.
    using C = Attend<D, F8, MT, PG16>;
    const sv_cache& c = a.cache;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, g = lane >> 4;
    // grid: slot blocks fastest, then kv heads, requests and parts
    int id = spread(block, blocks, a.xcd_run * a.slot_blocks);
    const int mb = id % a.slot_blocks;
    id /= a.slot_blocks;
    const int h = id % c.n_kv_heads;
    id /= c.n_kv_heads;
    int r = id % a.n_req;
    const int part = id / a.n_req;
    if (a.longest_first) r = longest(r, a.ctx_len, a.n_req, sm.lens);

    const int lo = a.cu_rows[r], hi = a.cu_rows[r + 1];
    const int rows = hi - lo;
    if (lo < 0 || hi < lo || rows > a.k_max + 1 || hi > a.q_rows) {
        if (threadIdx.x == 0) raise_error(a.dev_error, SV_DEV_BAD_CU_ROWS);
        return;
    }
    const int ctx = a.ctx_len[r];
    const int first = OWN ? a.first[r] : 0;
    if (OWN && first < 0) return;
    if (ctx < first || (int64_t)ctx + rows > (int64_t)a.max_pages * c.page_size) {
        if (threadIdx.x == 0) raise_error(a.dev_error, SV_DEV_BAD_CTX);
        return;
    }
    const int G = a.group;
    const int slots = rows * G - mb * 16 * MT;  // slots of this block
    if (slots <= 0) return;
    const int len = ctx + rows;
    const int base = OWN ? first & ~15 : 0;  // tiles' halves lie in one page
    const int plen = part_len(len - base, a.parts, a.part_min);
    const int begin = base + part * plen, end = min(len, begin + plen);
    if (begin >= len) return;
    const bool whole = !OWN && plen >= len;  // the request's only part

    const char* kbase = static_cast<const char*>(c.k) + (int64_t)h * c.head_stride * C::kEsize;
    const char* vbase = static_cast<const char*>(c.v) + (int64_t)h * c.head_stride * C::kEsize;
    const int32_t* table = a.page_table + (int64_t)r * a.max_pages;
    // Byte offset of position t's row.  A bad page id is reported and its
    // positions count as absent (ok = false); the offset then is page 0's.
    auto row_offset = [&](int t, bool& ok) -> int64_t {
        t = min(t, len - 1);
        if (OWN) t = max(t, first);  // the prefix's pages need not be the request's
        int page = table[t / c.page_size];
        ok = page >= 0 && page < c.n_pages;
        page = ok ? page : 0;
        return ((int64_t)page * c.page_stride + (int64_t)(t % c.page_size) * c.token_stride) *
               C::kEsize;
    };
    // Pages of a multiple of 16 positions hold each half of a tile (16
    // positions) in one page: two ids a tile, the same in every lane, fetched
    // a tile ahead of the loads that need them.
    const int last16 = (len - 1) & ~15;
    auto page_index = [&](int t) {
        return a.page_shift >= 0 ? t >> a.page_shift : (int)((unsigned)t / (unsigned)c.page_size);
    };
    struct Ids {
        int page[C::kHalves];
    };
    auto look_up = [&](int t0) {
        Ids p;
#pragma unroll
        for (int u = 0; u < C::kHalves; ++u)
            p.page[u] = table[page_index(min(t0 + 16 * u, last16))];
        return p;
    };

    Words<4> kr[C::kHalves][C::kKLoads];
    const int64_t tstride = c.token_stride * C::kEsize;
    const uint32_t koff = (uint32_t)(col * tstride) + g * 16;
    const uint32_t voff = (uint32_t)(g * 4 * tstride) + col * C::kDpl * C::kEsize;
    struct Values {
        Words<C::kVWords> r[4 * C::kHalves];
        uint32_t ok;  // bit j: the page of the lane's j-th position is good
    };
    Values vals;
    // Issues a tile's loads of keys or of values.
    auto load = [&](int t0, Ids ids, bool keys) __attribute__((always_inline)) {
        if (PG16) {
            const char* at[C::kHalves];
            uint32_t ok = 0;
#pragma unroll
            for (int u = 0; u < C::kHalves; ++u) {
                const int t = min(t0 + 16 * u, last16);
                int page = __builtin_amdgcn_readfirstlane(ids.page[u]);
                const bool good = page >= 0 && page < c.n_pages;
                ok |= good ? 0xfu << (4 * u) : 0u;
                page = good ? page : 0;
                const int slot = t - page_index(t) * c.page_size;
                const int64_t off =
                    ((int64_t)page * c.page_stride + (int64_t)slot * c.token_stride) * C::kEsize;
                at[u] = (keys ? kbase : vbase) + off;
            }
            if (keys) {
#pragma unroll
                for (int u = 0; u < C::kHalves; ++u)
#pragma unroll
                    for (int i = 0; i < C::kKLoads; ++i)
                        kr[u][i] = load_words<4>(at[u] + (koff + i * 64));
            } else {
                vals.ok = ok;
#pragma unroll
                for (int j = 0; j < 4 * C::kHalves; ++j)
                    vals.r[j] = load_words<C::kVWords>(at[j >> 2] +
                                                     (voff + (uint32_t)((j & 3) * tstride)));
            }
        } else if (keys) {
#pragma unroll
            for (int u = 0; u < C::kHalves; ++u) {
                bool ok;
                const char* at = kbase + row_offset(t0 + 16 * u + col, ok);
#pragma unroll
                for (int i = 0; i < C::kKLoads; ++i)
                    kr[u][i] = load_words<4>(at + (i * 64 + g * 16));
            }
        } else {
            vals.ok = 0;
#pragma unroll
            for (int j = 0; j < 4 * C::kHalves; ++j) {
                bool ok;
                const char* at = vbase + row_offset(t0 + 16 * (j >> 2) + g * 4 + (j & 3), ok);
                vals.ok |= ok ? 1u << j : 0u;
                vals.r[j] = load_words<C::kVWords>(at + col * C::kDpl * C::kEsize);
            }
        }
    };

    // the first tile's loads go out before anything else is done
    const int stride = C::kWaves * C::kTile;
    int t0 = begin + wave * C::kTile;
    Ids ids{};
    if (t0 < end) {
        if (PG16) ids = look_up(t0);
        load(t0, ids, true);
        load(t0, ids, false);
        if (PG16) ids = look_up(min(t0 + stride, len - 1));
    }

    // queries of the block's slots: wave w brings steps w, w + 4, ...
    const uint16_t* qp = static_cast<const uint16_t*>(a.q);
    int last[MT];  // the last position the lane's slot sees
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const int i = mt * 16 + col, slot = mb * 16 * MT + i;
        const bool live = i < slots;
        const int row = slot / G, head = h * G + slot % G;
        last[mt] = live ? ctx + row : -1;
        for (int st = wave; st < C::kSteps; st += C::kWaves) {
            const int d = F8 ? (st / 2) * 64 + g * 16 + (st & 1) * 8 : st * 32 + g * 8;
            uint4 w = make_uint4(0, 0, 0, 0);
            if (live)
                w = *reinterpret_cast<const uint4*>(qp + (int64_t)(lo + row) * a.q_ld +
                                                    (int64_t)head * D + d);
            sm.q[mt][st][lane] = w;
        }
    }
    __syncthreads();
    const float scale =
        a.scale * kLog2e * (F8 && c.k_scale != nullptr ? c.k_scale[h] : 1.0f);

    f32x4 acc[MT][C::kDpl];
    float m[MT], mu[MT], l[MT];  // running m (-inf: no score yet), the m used, sum
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
        for (int i = 0; i < C::kDpl; ++i) acc[mt][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        m[mt] = -kInf;
        mu[mt] = 0.0f;
        l[mt] = 0.0f;
    }
    int bad = 0;

    while (t0 < end) {
        constexpr int U = C::kHalves, J = 4 * U;  // halves; positions a lane holds
        constexpr uint32_t kAllOk = (1u << J) - 1;
        f32x4 s[MT][U];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int u = 0; u < U; ++u) s[mt][u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int st = 0; st < C::kSteps; ++st) {
            bf16x8 k8[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (F8) {
                    const uint32_t w0 = kr[u][st / 2].w[(st & 1) * 2];
                    const uint32_t w1 = kr[u][st / 2].w[(st & 1) * 2 + 1];
                    k8[u] = as_bf16x8(e4m3_pair<false>(w0), e4m3_pair<true>(w0),
                                      e4m3_pair<false>(w1), e4m3_pair<true>(w1));
                } else {
                    const Words<4>& w = kr[u][F8 ? 0 : st];
                    k8[u] = as_bf16x8(w.w[0], w.w[1], w.w[2], w.w[3]);
                }
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                const uint4 w = sm.q[mt][st][lane];
                const bf16x8 q8 = as_bf16x8(w.x, w.y, w.z, w.w);
#pragma unroll
                for (int u = 0; u < U; ++u)
                    s[mt][u] =
                        __builtin_amdgcn_mfma_f32_16x16x32_bf16(k8[u], q8, s[mt][u], 0, 0, 0);
            }
        }
        // the next tile's keys, in flight over the softmax and the product with
        // the values (the scores are taken first: the keys' registers); its
        // values follow the product, into the same registers.  A second set of
        // value registers spills: 445 us of 256 requests against 394.
        const int t1 = t0 + stride;
        const bool more = t1 < end;
        const Ids ids1 = ids;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int u = 0; u < U; ++u) asm volatile("" : "+v"(s[mt][u]));
        if (more) {
            load(t1, ids1, true);
            if (PG16) ids = look_up(min(t1 + stride, len - 1));
        }
        __builtin_amdgcn_sched_barrier(0);

        // Positions past the context are not seen by every row; positions past
        // the end, or on a bad page, by none: their values are zeroed, since 0
        // times what lies there may be NaN.  A value that is not finite behind
        // the context poisons the product for the rows that do not see it.
        if (vals.ok != kAllOk) bad = 1;
        const bool edge = t0 + C::kTile > ctx || __ballot(vals.ok != kAllOk) != 0 ||
                          (OWN && t0 < first);
        bool poison = false;
        if (edge) {
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const int t = t0 + 16 * (j >> 2) + g * 4 + (j & 3);
                const bool in = t < len && ((vals.ok >> j) & 1) && (!OWN || t >= first);
                bool nf = false;
#pragma unroll
                for (int i = 0; i < C::kVWords; ++i) {
                    if (!in) vals.r[j].w[i] = 0;
                    if (F8) {
                        nf |= bf16_pair_nonfinite(e4m3_pair<false>(vals.r[j].w[i])) ||
                              bf16_pair_nonfinite(e4m3_pair<true>(vals.r[j].w[i]));
                    } else {
                        nf |= bf16_pair_nonfinite(vals.r[j].w[i]);
                    }
                }
                poison |= nf && t > ctx;
            }
            poison = __ballot(poison) != 0;
        }
        bf16x8 pb[MT], pr[MT];  // the weights' upper halves and rests
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            if (mt * 16 >= slots) break;
            float p[J];
#pragma unroll
            for (int j = 0; j < J; ++j) p[j] = s[mt][j >> 2][j & 3] * scale;
            if (edge) {
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    const int t = t0 + 16 * (j >> 2) + g * 4 + (j & 3);
                    if (t > last[mt] || !((vals.ok >> j) & 1) || (OWN && t < first)) p[j] = -kInf;
                }
            }
            float mx = p[0];
#pragma unroll
            for (int j = 1; j < J; ++j) mx = fmaxf(mx, p[j]);
            // m moves only when a score passes the maximum it came from by 2^8,
            // or the sum is full: sums and outputs are relative to it either
            // way; most tiles then rescale nothing
            if (__ballot(mx > m[mt] + (8.0f - C::kHold) || (!F8 && l[mt] > C::kFull)) != 0) {
                mx = fmaxf(mx, __shfl_xor(mx, 16));
                mx = fmaxf(mx, __shfl_xor(mx, 32));
                float to = fmaxf(m[mt], mx + C::kHold);
                if (!F8) {
                    float most = fmaxf(l[mt], __shfl_xor(l[mt], 16));
                    most = fmaxf(most, __shfl_xor(most, 32));
                    if (most > C::kFull) to += C::kRaise;
                }
                if (to > m[mt]) {
                    const float f = fast_exp2(m[mt] - to);  // m = -inf: 0
#pragma unroll
                    for (int i = 0; i < C::kDpl; ++i) acc[mt][i] *= f;
                    l[mt] *= f;
                    m[mt] = mu[mt] = to;
                }
            }
#pragma unroll
            for (int j = 0; j < J; ++j) {
                p[j] = fast_exp2(p[j] - mu[mt]);
                l[mt] += p[j];
            }
            // Weights go into the matrix product as two bf16 terms, the upper
            // half of the fp32 weight and the rest, off by at most 2^-15 of each.
            // Both are positive where the weight is (the rest of 1 + 2^-23 times
            // it is taken): an infinite value times 0 or a negative rest would
            // make NaN.  One term (2^-8) let the error against 64 bits grow by up
            // to a quarter; the second costs 0 .. 2 % where reading bounds the
            // call (256 requests, ctx 4096: 392.0 and 393.7 us; 3 x 100,005 e4m3:
            // 141.4 and 144.8), 8 % at four slot tiles.
            constexpr float kOneUp = 1.0f + 0x1p-23f;
            uint32_t hw[4], rw[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t a = __float_as_uint(p[2 * i]), b = __float_as_uint(p[2 * i + 1]);
                hw[i] = __builtin_amdgcn_perm(b, a, 0x07060302u);
                rw[i] = pack_bf16(fmaf(p[2 * i], kOneUp, -bf16_hi(a)),
                                  fmaf(p[2 * i + 1], kOneUp, -bf16_hi(b)));
            }
            pb[mt] = as_bf16x8(hw[0], hw[1], hw[2], hw[3]);
            pr[mt] = as_bf16x8(rw[0], rw[1], rw[2], rw[3]);
            if (poison) {
                // position by position, each row only what it sees
                for (int gg = 0; gg < 4; ++gg) {
#pragma unroll
                    for (int j = 0; j < J; ++j) {
                        const float pj = __shfl(p[j], gg * 16 + col);
                        const int t = t0 + 16 * (j >> 2) + gg * 4 + (j & 3);
                        bool ok;
                        const char* at = vbase + row_offset(t, ok) + g * C::kAcc * C::kEsize;
                        if (t > last[mt] || t >= len || !ok || (OWN && t < first)) continue;
#pragma unroll
                        for (int e = 0; e < C::kAcc; ++e) {
                            float v;
                            if (F8) {
                                const uint32_t w = reinterpret_cast<const uint8_t*>(at)[e];
                                v = __uint_as_float(e4m3_pair<false>(w) << 16);
                            } else {
                                v = __uint_as_float(
                                    (uint32_t)reinterpret_cast<const uint16_t*>(at)[e] << 16);
                            }
                            acc[mt][e % C::kDpl][e / C::kDpl] += pj * v;
                        }
                    }
                }
            }
        }
        if (!poison) {
#pragma unroll
            for (int i2 = 0; i2 < C::kDpl / 2; ++i2) {
                uint32_t w[8];  // dims 2 i2 and 2 i2 + 1 of the lane's 8 positions
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const Words<C::kVWords>& v = vals.r[j];
                    if (F8)
                        w[j] = (i2 & 1) ? e4m3_pair<true>(v.w[i2 / 2])
                                        : e4m3_pair<false>(v.w[i2 / 2]);
                    else
                        w[j] = v.w[F8 ? 0 : i2];
                }
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const uint32_t sel = half ? 0x07060302u : 0x05040100u;
                    const bf16x8 vt = as_bf16x8(__builtin_amdgcn_perm(w[1], w[0], sel),
                                                __builtin_amdgcn_perm(w[3], w[2], sel),
                                                __builtin_amdgcn_perm(w[5], w[4], sel),
                                                __builtin_amdgcn_perm(w[7], w[6], sel));
                    const int i = 2 * i2 + half;
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        if (mt * 16 >= slots) break;
                        acc[mt][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vt, pb[mt],
                                                                             acc[mt][i], 0, 0, 0);
                        acc[mt][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vt, pr[mt],
                                                                             acc[mt][i], 0, 0, 0);
                    }
                }
            }
        }
        if (more) load(t1, ids1, false);
        t0 = t1;
    }
    if (__ballot(bad) != 0 && lane == 0) raise_error(a.dev_error, SV_DEV_BAD_PAGE);

    // sums over the four lane groups of a slot
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        l[mt] += __shfl_xor(l[mt], 16);
        l[mt] += __shfl_xor(l[mt], 32);
    }
    // the waves' results, two by two: 2, 3 into 0, 1, then 1 into 0
#pragma unroll
    for (int round = 0; round < 2; ++round) {
        const int from = round == 0 ? 2 : 1, n = round == 0 ? 2 : 1;
        __syncthreads();
        if (wave >= from && wave < from + n) {
            const int b = wave - from;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                if (mt * 16 >= slots) break;
#pragma unroll
                for (int i = 0; i < C::kDpl; ++i)
                    *reinterpret_cast<f32x4*>(sm.part.acc[b][mt][i][lane]) = acc[mt][i];
                sm.part.m[b][mt][lane] = m[mt];
                sm.part.l[b][mt][lane] = l[mt];
            }
        }
        __syncthreads();
        if (wave < n) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                if (mt * 16 >= slots) break;
                const float m2 = sm.part.m[wave][mt][lane], l2 = sm.part.l[wave][mt][lane];
                const float mx = fmaxf(m[mt], m2);
                const float f1 = m[mt] == mx ? 1.0f : fast_exp2(m[mt] - mx);
                const float f2 = m2 == mx ? 1.0f : fast_exp2(m2 - mx);
                l[mt] = l[mt] * f1 + l2 * f2;
                m[mt] = mx;
#pragma unroll
                for (int i = 0; i < C::kDpl; ++i) {
                    const f32x4 o = *reinterpret_cast<const f32x4*>(sm.part.acc[wave][mt][i][lane]);
                    acc[mt][i] = acc[mt][i] * f1 + o * f2;
                }
            }
        }
    }
    if (wave != 0) return;

    const float vscale = F8 && c.v_scale != nullptr ? c.v_scale[h] : 1.0f;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const int i = mt * 16 + col, slot = mb * 16 * MT + i;
        if (i >= slots) continue;
        const int row = slot / G, head = h * G + slot % G;
        if (whole) {
            // no weight at all: 0, also where 0 times a value was NaN
            if (l[mt] == 0.0f) {
#pragma unroll
                for (int e = 0; e < C::kDpl; ++e) acc[mt][e] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            }
            // the mean first, then its scale: only their product has to be in range
            const float inv = l[mt] == 0.0f ? 0.0f : 1.0f / l[mt];
            uint32_t w[C::kAcc / 2];
#pragma unroll
            for (int e = 0; e < C::kAcc; e += 2)
                w[e / 2] =
                    pack_bf16(acc[mt][e % C::kDpl][e / C::kDpl] * inv * vscale,
                              acc[mt][(e + 1) % C::kDpl][(e + 1) / C::kDpl] * inv * vscale);
            uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) +
                                                (int64_t)(lo + row) * a.out_ld +
                                                (int64_t)head * D + g * C::kAcc);
#pragma unroll
            for (int e = 0; e < C::kAcc / 8; ++e)
                o[e] = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
            if (a.out_lse != nullptr && g == 0)
                a.out_lse[(int64_t)(lo + row) * a.n_heads + head] =
                    l[mt] == 0.0f
                        ? -kInf
                        : ((m[mt] - C::kHold) + log2f(l[mt] * exp2f(C::kHold))) * kLn2;
        } else {
            const int64_t rec = (((int64_t)r * a.n_heads + head) * (a.k_max + 1) + row) * a.parts +
                                part;
            f32x4* o = reinterpret_cast<f32x4*>(a.part_out + rec * D + g * C::kAcc);
#pragma unroll
            for (int e = 0; e < C::kAcc; e += 4) {
                f32x4 x;
#pragma unroll
                for (int i4 = 0; i4 < 4; ++i4)
                    x[i4] = acc[mt][(e + i4) % C::kDpl][(e + i4) / C::kDpl];
                o[e / 4] = x;
            }
            if (g == 0) {
                a.part_ml[rec * 2] = m[mt];
                a.part_ml[rec * 2 + 1] = l[mt];
            }
        }
    }
