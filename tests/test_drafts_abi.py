"""Host-side refusals of the drafted-token operators (tree attention, batched prep, cache read and
commit): every bad argument is an error code before anything is launched (no GPU needed)."""
import ctypes

import pytest

from int8_kv_top_gb300 import build as qbuild
from int8_kv_top_gb300 import qsa

FAKE = 1 << 20  # aligned, never dereferenced: every call below fails validation first
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return qsa.load()


def call(fn, args, **over):
    """fn with `args` (an ordered dict of valid arguments), some of them replaced."""
    unknown = set(over) - set(args)
    assert not unknown, unknown
    return fn(*[over.get(k, v) for k, v in args.items()])


PREP = dict(q_raw=P(FAKE), k_raw=P(FAKE), v_raw=P(FAKE), q_stride=6144, k_stride=512, v_stride=512, q_gamma=P(FAKE),
            k_gamma=P(FAKE), pos=P(FAKE), axes=1, cells=P(FAKE), rope=None, n_tok=4, n_pool=100, qcur=P(FAKE), kcur=None,
            kq=P(FAKE), ksc=P(FAKE), vq=P(FAKE), vsc=P(FAKE), stream=None)
READ = dict(kq=P(FAKE), ksc=P(FAKE), vq=P(FAKE), vsc=P(FAKE), n_pool=100, cells=P(FAKE), n=4, k16=P(FAKE), v16=P(FAKE),
            stream=None)
TREE = dict(q=P(FAKE), kq=P(FAKE), vq=P(FAKE), ksc=P(FAKE), vsc=P(FAKE), n_pool=100, seqs=P(FAKE), n_seq=1, n_tok=4,
            tree=P(FAKE), tree_words=1, max_n_kv=50, ids=None, gate=None, out=P(FAKE), ws=None, ws_bytes=0, params=None,
            stream=None)
COMMIT = dict(kq=P(FAKE), ksc=P(FAKE), vq=P(FAKE), vsc=P(FAKE), n_pool=100, seqs=P(FAKE), n_seq=2, path=P(FAKE),
              n_path=P(FAKE), path_cap=4, stream=None)
FNS = {"qsa_prep_batched": PREP, "qsa_cache_read": READ, "qsa_tree_attention": TREE, "qsa_cache_commit": COMMIT}
OPTIONAL = {"kcur", "rope", "stream", "ids", "gate", "ws", "params", "k16", "v16"}


@pytest.mark.parametrize("name", list(FNS))
def test_null_and_misaligned_pointers(lib, name):
    fn, args = getattr(lib, name), FNS[name]
    for k, v in args.items():
        if not isinstance(v, P):
            continue
        assert call(fn, args, **{k: P(FAKE + 8)}) == qsa.QSA_ERR_INVALID_ARG, k
        assert b"aligned" in lib.qsa_last_error() and k.encode() in lib.qsa_last_error()
        if k not in OPTIONAL:
            assert call(fn, args, **{k: None}) == qsa.QSA_ERR_INVALID_ARG, k
            assert b"NULL" in lib.qsa_last_error()
    for k in ("kcur", "ids", "gate", "ws"):
        if k in args:
            assert call(fn, args, **{k: P(FAKE + 4)}) == qsa.QSA_ERR_INVALID_ARG, k


@pytest.mark.parametrize("name", list(FNS))
@pytest.mark.parametrize("n_pool", [0, -1, 1 << 31, 1 << 40])
def test_pool_sizes(lib, name, n_pool):
    assert call(getattr(lib, name), FNS[name], n_pool=n_pool) == qsa.QSA_ERR_INVALID_ARG
    assert b"n_pool" in lib.qsa_last_error()


def test_nothing_to_do_is_no_error(lib):
    null = dict.fromkeys(("q_raw", "kq", "ksc", "vq", "vsc", "cells", "qcur"), None)
    assert call(lib.qsa_prep_batched, PREP, n_tok=0, **null) == qsa.QSA_OK
    assert call(lib.qsa_cache_read, READ, n=0, kq=None, cells=None) == qsa.QSA_OK
    assert call(lib.qsa_tree_attention, TREE, n_tok=0, n_seq=0, q=None, out=None) == qsa.QSA_OK
    assert call(lib.qsa_cache_commit, COMMIT, n_seq=0, kq=None, path=None) == qsa.QSA_OK


def test_prep_batched_refusals(lib):
    f = lib.qsa_prep_batched
    assert call(f, PREP, n_tok=-1) == qsa.QSA_ERR_INVALID_ARG
    for axes in (0, 2, 4):
        assert call(f, PREP, axes=axes) == qsa.QSA_ERR_INVALID_ARG
    for k, w in (("q_stride", 6144), ("k_stride", 512), ("v_stride", 512)):
        for bad in (w - 8, w + 4, 0, -w):
            assert call(f, PREP, **{k: bad}) == qsa.QSA_ERR_INVALID_ARG
            assert k.encode() in lib.qsa_last_error()

    def rope(base=10000.0, rd=256, eps=1e-6, sec=(32, 48, 48)):
        return ctypes.byref(qsa.qsa_rope(base, rd, eps, (ctypes.c_int * 3)(*sec)))

    for rd in (8, 24, 512, 0):
        assert call(f, PREP, rope=rope(rd=rd)) == qsa.QSA_ERR_UNSUPPORTED
    for base in (1.0, 0.0, float("inf"), float("nan")):
        assert call(f, PREP, rope=rope(base=base)) == qsa.QSA_ERR_INVALID_ARG
    for eps in (0.0, -1e-6, 1.0, float("nan")):
        assert call(f, PREP, rope=rope(eps=eps)) == qsa.QSA_ERR_INVALID_ARG
    for sec in ((32, 48, 47), (-1, 65, 64), (2**31 - 1, 2**31 - 1, 130)):
        assert call(f, PREP, axes=3, rope=rope(sec=sec)) == qsa.QSA_ERR_INVALID_ARG


def test_cache_read_refusals(lib):
    assert call(lib.qsa_cache_read, READ, n=-1) == qsa.QSA_ERR_INVALID_ARG
    assert call(lib.qsa_cache_read, READ, k16=None, v16=None) == qsa.QSA_ERR_INVALID_ARG


def test_tree_attention_refusals(lib):
    f = lib.qsa_tree_attention
    assert call(f, TREE, n_tok=-1) == qsa.QSA_ERR_INVALID_ARG
    assert call(f, TREE, n_seq=-1) == qsa.QSA_ERR_INVALID_ARG
    assert call(f, TREE, max_n_kv=0) == qsa.QSA_ERR_INVALID_ARG
    assert call(f, TREE, n_tok=65536) == qsa.QSA_ERR_UNSUPPORTED
    assert call(f, TREE, n_seq=65536) == qsa.QSA_ERR_UNSUPPORTED
    for w in (0, -1, 9):
        assert call(f, TREE, tree_words=w) == qsa.QSA_ERR_UNSUPPORTED
    for bad in (qsa.qsa_params(0, 2051, 0.0625), qsa.qsa_params(2053, 2051, 0.0625), qsa.qsa_params(8, 0, 0.0625),
                qsa.qsa_params(8, 20, -1.0), qsa.qsa_params(8, 20, float("nan"))):
        assert call(f, TREE, params=ctypes.byref(bad)) == qsa.QSA_ERR_INVALID_ARG
        assert qsa.qsa_tree_attention_workspace_bytes(1, 4, 50, bad) == 0
    need = qsa.qsa_tree_attention_workspace_bytes(3, 40, 9000)
    if need:  # a call whose workspace is missing or short by a byte
        big = dict(TREE, n_pool=40000, n_seq=3, n_tok=40, max_n_kv=9000)
        assert call(f, big) == qsa.QSA_ERR_WORKSPACE
        assert call(f, big, ws=P(FAKE), ws_bytes=need - 1) == qsa.QSA_ERR_WORKSPACE
    for args in ((0, 4, 50), (1, 0, 50), (1, 4, 0), (-1, 4, 50)):
        assert qsa.qsa_tree_attention_workspace_bytes(*args) == 0


def test_cache_commit_refusals(lib):
    assert call(lib.qsa_cache_commit, COMMIT, n_seq=-1) == qsa.QSA_ERR_INVALID_ARG
    for cap in (0, -3):
        assert call(lib.qsa_cache_commit, COMMIT, path_cap=cap) == qsa.QSA_ERR_INVALID_ARG
