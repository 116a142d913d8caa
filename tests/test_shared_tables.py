"""Where the launches of qsa_prefix_attention read and write for tables of any contents, as their own index arithmetic has it
(csrc/tree_tables.cuh, compiled for the host): rows of scores and of selected cells, and the parts that the join reads."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

from int8_kv_top_gb300 import build as qbuild

SHIM = r'''
#include <algorithm>
#include <cstdint>
#include <vector>
#define __device__
#define __forceinline__ inline
using std::max;
using std::min;
struct int4 { int x, y, z, w; };
static int4 make_int4(int x, int y, int z, int w) { return {x, y, z, w}; }
template <class T> static T __ldg(const T* p) { return *p; }
template <class T> static T __ldcg(const T* p) { return *p; }
static int __popc(unsigned x) { return __builtin_popcount(x); }
#include "tree_plan.cuh"
namespace qsa { constexpr int kHPG = kPlanHeads, kGroups = kPlanGroups, kTreeWords = 8; }
#include "tree_tables.cuh"

using namespace qsa;
static int up(int x, int to) { return (x + to - 1) / to * to; }

// 0: all inside.  1, 2: a score of a prefix, an own cell is stored past its row.  3, 4: bits past it are read.  5, 6: parts
// that are not there are read.  7: a record that is not its sequence's.
extern "C" int outside(const int4* seqs, int n_seq, const int4* prefixes, int n_prefix, int n_tok, int max_prefix, int max_n_kv,
                       int identity_max, long long n_pool, int clusters, int own_runs, int* valid) {
  TreeBatch b{seqs, n_pool, n_seq, n_tok, nullptr, 0, max_n_kv, identity_max};
  b.prefixes = prefixes;
  b.n_prefix = n_prefix;
  b.max_prefix = max_prefix;
  std::vector<int4> tok(n_tok);
  std::vector<TokMore> more(n_tok);
  b.tok = tok.data();
  *valid = 0;
  for (int t = 0; t < n_tok; ++t) {
    const int s = last_at(n_seq, t, [&](int i) { return seqs[i].w; });
    tok[t] = shared_record(b, t, s, prefix_of(b, s), &more[t]);
    *valid += tok[t].x >= 0;
  }
  const int pitch = up(max_n_kv + 127, 256);
  for (CellsOf of : {kPrefixCells, kOwnCells})
    for (int i = 0; i < (of == kPrefixCells ? n_prefix : n_seq); ++i) {
      int4 e;
      const int T = of == kPrefixCells ? prefix_tokens(b, i, &e) : shared_seq_tokens(b, i, &e);
      const int cells = of == kPrefixCells ? e.y : e.z + T, behind = of == kPrefixCells ? 0 : shared_seq(b, i, prefix_of(b, i)).pe.y;
      for (int k = 0; k < T; ++k) {
        const int4 ti = record_in(b, of, i, e.w + k);
        if (ti.x < 0 || ti.y <= identity_max) continue;
        if (score_column(of, behind) + (of == kPrefixCells ? up(cells, kTileCells) : cells) > pitch) return of == kPrefixCells ? 1 : 2;
        if ((of == kPrefixCells ? 0 : own_column(ti.z)) + up(cells, kTileCells) > pitch) return of == kPrefixCells ? 3 : 4;
      }
    }
  // the prefixes' clusters, a run each (or, of one prefix, as many as there are)
  std::vector<int4> plan;
  int at = 0;
  for (int p = 0; p < n_prefix; ++p) {
    int4 e;
    const int T = max(prefix_tokens(b, p, &e), 0), n = T > 0 && e.y > 0 ? up(T * kHPG, kTreeBlock) / kTreeBlock * kGroups : 0;
    plan.push_back(n_prefix == 1 ? only_prefix_plan(e.w, T, e.y, clusters) : make_int4(at, n > 0 && at + n <= clusters, e.w, T));
    at += n;
  }
  for (int t = 0; t < n_tok; ++t) {
    const int4 ti = tok[t], e = more[t].seq;
    if (ti.x < 0) continue;
    if (t < e.w || t >= e.w + e.z || ti.x >= n_seq) return 7;
    for (int h = 0; h < kHPG; ++h)
      for (int g = 0; g < kGroups; ++g) {
        size_t cta;
        int row;
        if (ti.z > 0 && plan[ti.w].y > 0) {
          const int4 pl = plan[ti.w];
          const long long R = (long long)(t - pl.z) * kHPG + h;
          if (R < 0 || R >= (long long)pl.w * kHPG) return 5;
          part_row(pl.x, pl.w, g, pl.y, (int)R, &cta, &row);
          if (cta + 2 * (pl.y - 1) >= (size_t)clusters * 2 || row < 0 || row >= kTreeBlock / 2) return 5;
        }
        part_row(first_block(e.w, ti.x) * kGroups * own_runs, e.z, g, own_runs, (t - e.w) * kHPG + h, &cta, &row);
        if (cta + 2 * (own_runs - 1) >= (size_t)tree_blocks_most(n_seq, n_tok) * kGroups * own_runs * 2 || row < 0 || row >= kTreeBlock / 2)
          return 6;
      }
  }
  return 0;
}

extern "C" int pairs(int n_prefix, int n_tok) { return tree_blocks_most(n_prefix, n_tok) * kPlanGroups; }
'''


@pytest.fixture(scope="module")
def outside(tmp_path_factory):
    d = tmp_path_factory.mktemp("tables")
    (d / "t.cpp").write_text(SHIM)
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-I", qbuild.CSRC, "-o", str(d / "t.so"), str(d / "t.cpp")], check=True)
    lib = ctypes.CDLL(str(d / "t.so"))

    def call(seqs, prefixes, n_tok, max_prefix, max_n_kv, identity_max=71, n_pool=1 << 30, clusters=0, own_runs=1):
        seqs, prefixes = (np.ascontiguousarray(x, np.int32).reshape(-1, 4) for x in (seqs, prefixes))
        valid = ctypes.c_int()
        clusters = max(clusters, lib.pairs(len(prefixes), n_tok))
        bad = lib.outside(seqs.ctypes.data_as(ctypes.c_void_p), len(seqs), prefixes.ctypes.data_as(ctypes.c_void_p), len(prefixes), n_tok,
                          max_prefix, max_n_kv, identity_max, ctypes.c_longlong(n_pool), clusters, own_runs, ctypes.byref(valid))
        return bad, valid.value

    return call


def table(rng, n_seq, n_prefix, tokens):
    """A valid table, in which long prefixes and long own runs come apart, and its bounds."""
    t = rng.integers(0, tokens + 1, n_seq)
    t[rng.integers(n_seq)] += 1
    starts = np.concatenate([[0], np.sort(rng.integers(0, n_seq + 1, max(n_prefix - 1, 0)))])[:n_prefix]
    shared = rng.choice([0, 5, 128, 3000, 30000], n_prefix)
    mine = np.searchsorted(starts, np.arange(n_seq), side="right") - 1
    behind = shared[mine] if n_prefix else np.zeros(n_seq, int)
    held = np.where(behind >= 3000, rng.integers(0, 200, n_seq), rng.choice([0, 40, 2000, 32000], n_seq))
    seqs = np.stack([np.zeros(n_seq, int), held + t + 1, held, np.concatenate([[0], np.cumsum(t)[:-1]])], 1)
    prefixes = np.stack([np.zeros(n_prefix, int), shared, starts, np.zeros(n_prefix, int)], 1)
    return seqs, prefixes, int(t.sum()), int(max(shared, default=0)), int((behind + held + t).max())


def shapes(rng, n):
    for _ in range(n):
        n_seq = int(rng.choice([1, 2, 3, 8, 40, 120]))
        yield table(rng, n_seq, int(rng.choice([0, 1, 2, 3, 6])), int(rng.choice([1, 2, 6, 40, 200])))


def test_valid_tables_stay_inside(outside):
    rng = np.random.default_rng(1)
    for seqs, prefixes, n_tok, max_prefix, max_n_kv in shapes(rng, 400):
        bad, valid = outside(seqs, prefixes, n_tok, max_prefix, max_n_kv, clusters=int(rng.integers(1, 400)), own_runs=int(rng.integers(1, 9)))
        assert bad == 0 and valid == n_tok


def test_first_rows_that_run_backwards_store_and_read_inside(outside):
    # a token between two sequences that both name its row: one behind 30,000 cells, the other with 33,000 of its own
    seqs = [[0, 100, 2, 0], [0, 100, 2, 2], [0, 33000, 32990, 1]]
    assert outside(seqs, [[0, 30000, 0, 0], [0, 0, 1, 0]], 3, 30000, 33000, identity_max=2051)[0] in (0, 5, 6)


@pytest.mark.parametrize("how", ["rows in any order", "rows of any value", "first sequences too", "entries of any value"])
def test_broken_tables_store_and_read_rows_inside(outside, how):
    assert not broken(outside, how) & {1, 2, 3, 4, 7}


@pytest.mark.parametrize("how", ["rows in any order", "rows of any value", "first sequences too", "entries of any value"])
def test_broken_tables_join_parts_that_are_there(outside, how):
    assert broken(outside, how) == {0}


def broken(outside, how):
    """What is outside, over tables that break the contract."""
    rng = np.random.default_rng(7)
    seen, accepted = set(), 0
    for seqs, prefixes, n_tok, max_prefix, max_n_kv in shapes(rng, 1500):
        n_seq = len(seqs)
        if how == "rows of any value":
            seqs[1:, 3] = rng.integers(-5, n_tok + 6, n_seq - 1)
        elif how == "entries of any value":
            for x, most in ((seqs, max_n_kv), (prefixes, max_prefix)):
                if len(x):
                    x[rng.integers(len(x)), rng.integers(4)] = rng.choice([-2**31, -1, 0, 1, most, 2**31 - 1])
        else:
            seqs[1:, 3] = rng.permutation(seqs[1:, 3])
        if how == "first sequences too" and len(prefixes) > 1:
            prefixes[1:, 2] = rng.integers(-1, n_seq + 2, len(prefixes) - 1)
        bad, valid = outside(seqs, prefixes, n_tok, max_prefix, max_n_kv, clusters=int(rng.integers(1, 400)), own_runs=int(rng.integers(1, 9)))
        seen.add(bad)
        accepted += valid
    assert accepted > 1000
    return seen
