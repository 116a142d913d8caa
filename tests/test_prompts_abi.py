"""Host-side refusals of the operators for sequences that share a prompt, and what the binding looks at: every bad
argument is an error before anything is launched (no GPU needed)."""
import ctypes

import pytest
import torch

from int8_kv_top_gb300 import build as qbuild
from int8_kv_top_gb300 import qsa

FAKE = 1 << 20  # aligned, never dereferenced: every call below fails validation first
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return qsa.load()


def call(fn, args, **over):
    unknown = set(over) - set(args)
    assert not unknown, unknown
    return fn(*[over.get(k, v) for k, v in args.items()])


VERIFY = dict(p=P(FAKE), p_stride=100, d=P(FAKE), d_stride=100, vocab=100, token=P(FAKE), parent=P(FAKE), u=P(FAKE), u_end=P(FAKE),
              seqs=P(FAKE), n_seq=2, n_tok=8, path=P(FAKE), path_cap=4, n_path=P(FAKE), next=P(FAKE), stream=None)
COPY = dict(kq=P(FAKE), ksc=P(FAKE), vq=P(FAKE), vsc=P(FAKE), n_pool=100, runs=P(FAKE), n_run=3, max_cells=10, stream=None)
COMPACT = dict(kq=P(FAKE), ksc=P(FAKE), vq=P(FAKE), vsc=P(FAKE), n_pool=100, prefixes=P(FAKE), n_prefix=1, seqs=P(FAKE), n_seq=3,
               prefixes_out=P(FAKE), seqs_out=P(FAKE), used=P(FAKE), ws=P(FAKE), ws_bytes=1 << 20, stream=None)
ATTEND = dict(q=P(FAKE), kq=P(FAKE), vq=P(FAKE), ksc=P(FAKE), vsc=P(FAKE), n_pool=1000, prefixes=P(FAKE), n_prefix=1, seqs=P(FAKE),
              n_seq=2, n_tok=4, tree=P(FAKE), tree_words=1, max_prefix=100, max_n_kv=150, ids=P(FAKE), gate=P(FAKE), out=P(FAKE),
              ws=P(FAKE), ws_bytes=1 << 40, params=None, stream=None)
FNS = {"qsa_prefix_attention": ATTEND, "qsa_tree_verify": VERIFY, "qsa_cache_copy": COPY, "qsa_cache_compact": COMPACT}
MAY_BE_NULL = {"d", "used", "ws", "tree", "ids", "gate"}
ELEMENTS = {"p", "d", "token", "parent", "u", "u_end", "path", "n_path", "next", "used"}  # aligned to 4 bytes


@pytest.mark.parametrize("name", list(FNS))
def test_null_and_misaligned_pointers(lib, name):
    fn, args = getattr(lib, name), FNS[name]
    for k, v in args.items():
        if not isinstance(v, P):
            continue
        assert call(fn, args, **{k: P(FAKE + (2 if k in ELEMENTS else 8))}) == qsa.QSA_ERR_INVALID_ARG, k
        assert b"aligned" in lib.qsa_last_error() and k.encode() in lib.qsa_last_error()
        if k not in MAY_BE_NULL:
            assert call(fn, args, **{k: None}) == qsa.QSA_ERR_INVALID_ARG, k
            assert b"NULL" in lib.qsa_last_error()


@pytest.mark.parametrize("name", ["qsa_cache_copy", "qsa_cache_compact", "qsa_prefix_attention"])
@pytest.mark.parametrize("n_pool", [0, -1, 1 << 31, 1 << 40])
def test_pool_sizes(lib, name, n_pool):
    assert call(getattr(lib, name), FNS[name], n_pool=n_pool) == qsa.QSA_ERR_INVALID_ARG
    assert b"n_pool" in lib.qsa_last_error()


def test_nothing_to_do_is_no_error(lib):
    assert call(lib.qsa_tree_verify, VERIFY, n_seq=0, n_tok=0, p=None, seqs=None, path=None) == qsa.QSA_OK
    assert call(lib.qsa_cache_copy, COPY, n_run=0, kq=None, runs=None) == qsa.QSA_OK
    assert call(lib.qsa_cache_copy, COPY, max_cells=0, kq=None, runs=None) == qsa.QSA_OK
    assert call(lib.qsa_cache_compact, COMPACT, n_prefix=0, n_seq=0, kq=None, used=None, ws=None, ws_bytes=0) == qsa.QSA_OK


def test_attention_refusals(lib):
    f, size = lib.qsa_prefix_attention, qsa.qsa_prefix_attention_workspace_bytes
    assert call(f, ATTEND, n_tok=0, q=None) == call(f, ATTEND, n_seq=0, seqs=None) == qsa.QSA_OK
    for k in ("n_prefix", "n_seq", "n_tok"):
        assert call(f, ATTEND, **{k: -1}) == qsa.QSA_ERR_INVALID_ARG
        assert call(f, ATTEND, **{k: 65536}) == qsa.QSA_ERR_UNSUPPORTED
    for w in (0, -1, 9):
        assert call(f, ATTEND, tree_words=w) == qsa.QSA_ERR_UNSUPPORTED
    for over in (dict(max_n_kv=0, max_prefix=0), dict(max_prefix=-1)):
        assert call(f, ATTEND, **over) == qsa.QSA_ERR_INVALID_ARG
    assert call(f, ATTEND, max_n_kv=65410) == qsa.QSA_ERR_UNSUPPORTED
    assert call(f, ATTEND, max_prefix=(1 << 20) + 1) == qsa.QSA_ERR_UNSUPPORTED
    dense = qsa.qsa_params(2048, 1 << 21, 0.0625)
    assert call(f, ATTEND, max_n_kv=(1 << 20) + 1, params=ctypes.byref(dense)) == qsa.QSA_ERR_UNSUPPORTED
    for bad in (qsa.qsa_params(0, 2051, 0.0625), qsa.qsa_params(2053, 2051, 0.0625), qsa.qsa_params(8, 20, float("nan"))):
        assert call(f, ATTEND, params=ctypes.byref(bad)) == qsa.QSA_ERR_INVALID_ARG
        assert size(1, 2, 4, 100, 150, bad) == 0
    need = size(1, 2, 4, 100, 150)
    assert need > 0
    assert call(f, ATTEND, ws_bytes=need - 1) == qsa.QSA_ERR_WORKSPACE
    assert call(f, ATTEND, ws=None) == qsa.QSA_ERR_WORKSPACE
    for args in ((-1, 2, 4, 100, 150), (1, 0, 4, 100, 150), (1, 2, 0, 100, 150), (1, 2, 4, (1 << 20) + 1, 150), (1, 2, 4, 100, 0), (1, 2, 4, -1, 9)):
        assert size(*args) == 0


def test_attention_workspace_grows_with_each_argument(lib):
    import random
    rng = random.Random(1)
    size = qsa.qsa_prefix_attention_workspace_bytes
    for params in (None, (2048, 1 << 21, 0.0625)):
        for _ in range(400):
            a = [rng.choice((0, 1, 3, 70)), rng.choice((1, 2, 9, 64, 700)), rng.choice((1, 3, 8, 64, 300, 5000)), 0, 0]
            a[3] = rng.choice((0, 1, 127, 2000, 16000, 30000))
            a[4] = a[3] + rng.choice((1, 100, 2000, 30000))
            b = [x + rng.choice((0, 0, 1, 5, 300)) for x in a]
            b[4] = max(b[4], b[3])
            assert size(*a, params=params) <= size(*b, params=params), (a, b)


def test_verify_refusals(lib):
    f = lib.qsa_tree_verify
    for k in ("n_seq", "n_tok"):
        assert call(f, VERIFY, **{k: -1}) == qsa.QSA_ERR_INVALID_ARG
        assert call(f, VERIFY, **{k: 65536}) == qsa.QSA_ERR_UNSUPPORTED
    for vocab in (0, -5):
        assert call(f, VERIFY, vocab=vocab) == qsa.QSA_ERR_INVALID_ARG
    assert call(f, VERIFY, vocab=262145, p_stride=1 << 20, d_stride=1 << 20) == qsa.QSA_ERR_UNSUPPORTED
    for k in ("p_stride", "d_stride"):
        for bad in (99, 0, -100):
            assert call(f, VERIFY, **{k: bad}) == qsa.QSA_ERR_INVALID_ARG
            assert k.encode() in lib.qsa_last_error()
    for cap in (0, -1):
        assert call(f, VERIFY, path_cap=cap) == qsa.QSA_ERR_INVALID_ARG


def test_copy_refusals(lib):
    f = lib.qsa_cache_copy
    assert call(f, COPY, n_run=-1) == qsa.QSA_ERR_INVALID_ARG
    assert call(f, COPY, max_cells=-1) == qsa.QSA_ERR_INVALID_ARG
    assert call(f, COPY, n_run=65536) == qsa.QSA_ERR_UNSUPPORTED


def test_compact_refusals(lib):
    f, size = lib.qsa_cache_compact, qsa.qsa_cache_compact_workspace_bytes
    for k in ("n_prefix", "n_seq"):
        assert call(f, COMPACT, **{k: -1}) == qsa.QSA_ERR_INVALID_ARG
    assert call(f, COMPACT, n_prefix=30000, n_seq=40000) == qsa.QSA_ERR_UNSUPPORTED
    need = size(100, 1, 3)
    assert need > 0
    assert call(f, COMPACT, ws_bytes=need - 1) == qsa.QSA_ERR_WORKSPACE
    assert call(f, COMPACT, ws=None) == qsa.QSA_ERR_WORKSPACE
    for bad in ((0, 1, 1), (1 << 31, 1, 1), (100, -1, 1), (100, 1, -1), (100, 65535, 1)):
        assert size(*bad) == 0
    sizes = [size(p, a, b) for p, a, b in ((1, 1, 0), (100, 1, 0), (100, 1, 5), (5000, 1, 5), (5000, 7, 5), (10 ** 9, 535, 65000))]
    assert sizes == sorted(sizes)


# ---------------------------------------------------------------- the binding
N, V = 6, 40


class Fake:
    def __init__(self):
        self.calls = {}

    def __getattr__(self, name):
        return lambda *args: self.calls.__setitem__(name, args) or 0


@pytest.fixture
def fake(monkeypatch):
    f = Fake()
    monkeypatch.setattr(qsa, "load", lambda: f)
    monkeypatch.setattr(qsa, "_stream", lambda s=None: 0)
    return f.calls


def ints(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def refused(fn, *args, **kw):
    with pytest.raises(qsa.QSAError) as e:
        fn(*args, **kw)
    assert e.value.code == qsa.QSA_ERR_INVALID_ARG
    return str(e.value)


@pytest.mark.parametrize("name,bad", [("p", torch.zeros(N, V)), ("d", torch.zeros(N, V)), ("token", ints(N)), ("seqs", ints(2, 4))])
def test_tensors_that_are_not_on_the_gpu_are_refused(fake, name, bad):
    args = dict(p=FAKE, d=None, vocab=V, token=FAKE, parent=FAKE, u=FAKE, u_end=FAKE, seqs=FAKE, n_seq=2, n_tok=N, path=ints(2, 4),
                n_path=FAKE, next=FAKE)
    assert name in refused(qsa.qsa_tree_verify, **{**args, name: bad})
    assert fake == {}


def test_pools_and_tables_on_the_cpu_are_refused(fake):
    codes, scales = torch.zeros(9, 2, 256, dtype=torch.int8), torch.zeros(9, 2, 4, dtype=torch.float16)
    assert "kq" in refused(qsa.qsa_cache_copy, codes, scales, codes, scales, 9, ints(2, 4), 2, 5)
    assert "runs" in refused(qsa.qsa_cache_copy, FAKE, FAKE, FAKE, FAKE, 9, ints(2, 4), 2, 5)
    assert "prefixes" in refused(qsa.qsa_cache_compact, FAKE, FAKE, FAKE, FAKE, 9, ints(2, 4), 2, FAKE, 1, FAKE, FAKE, None, None)
    assert fake == {}


def test_absent_arrays_and_raw_pointers_pass(fake):
    qsa.qsa_cache_compact(FAKE, FAKE, FAKE, FAKE, 9, None, 0, FAKE, 2, None, FAKE, None, None)
    assert fake["qsa_cache_compact"] == (FAKE, FAKE, FAKE, FAKE, 9, None, 0, FAKE, 2, None, FAKE, None, None, 0, 0)
    assert "prefixes" in refused(qsa.qsa_cache_compact, FAKE, FAKE, FAKE, FAKE, 9, None, 1, FAKE, 2, None, FAKE, None, None)


def test_workspaces_on_the_cpu_are_refused(fake):
    assert "ws" in refused(qsa.qsa_cache_compact, FAKE, FAKE, FAKE, FAKE, 9, None, 0, FAKE, 2, None, FAKE, None, torch.zeros(99))
    assert "ws" in refused(qsa.qsa_prefix_attention, FAKE, FAKE, FAKE, FAKE, FAKE, 9, None, 0, FAKE, 2, 2, None, 0, 5, None, FAKE, torch.zeros(99))
    assert "path" in refused(qsa.qsa_tree_verify, FAKE, None, V, FAKE, FAKE, FAKE, FAKE, FAKE, 2, N, ints(8), FAKE, FAKE)
    assert fake == {}


def test_nothing_to_copy_in_a_pool_without_cells(lib):
    assert call(lib.qsa_cache_copy, COPY, n_pool=0, max_cells=0, kq=None, ksc=None, vq=None, vsc=None) == 0
    assert call(lib.qsa_cache_copy, COPY, n_pool=0) == qsa.QSA_ERR_INVALID_ARG


def test_masks_that_are_no_rows_of_words_are_refused(fake):
    for tree in (ints(2), ints(2, 1, 1), FAKE, [[1], [3]]):
        assert "tree" in refused(qsa.qsa_prefix_attention, FAKE, FAKE, FAKE, FAKE, FAKE, 9, None, 0, FAKE, 2, 2, tree, 0, 5, None, FAKE)
    assert fake == {}
