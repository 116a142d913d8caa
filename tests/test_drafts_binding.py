"""The Python binding of the drafted-token operators: what it reads as packed tables, and rows with a stride, is looked
at before a call (no GPU needed: every call below ends in its arguments, or in a fake of the library)."""
import pytest
import torch

from int8_kv_top_gb300 import qsa

N, POOL = 6, 100
FUSED = torch.zeros(N, 28 * 256, dtype=torch.float16)
Z = torch.zeros(1)


class Fake:
    """Stands for the library: records what the calls are given."""

    def __init__(self):
        self.calls = {}

    def __getattr__(self, name):
        return lambda *args: self.calls.__setitem__(name, args) or 0


@pytest.fixture
def lib(monkeypatch):
    fake = Fake()
    monkeypatch.setattr(qsa, "load", lambda: fake)
    monkeypatch.setattr(qsa, "_stream", lambda s=None: 0)
    return fake.calls


def ints(*shape, dtype=torch.int32):
    return torch.zeros(*shape, dtype=dtype)


def prep(n=N, q=FUSED[:, :6144], k=FUSED[:, 6144:6656], v=FUSED[:, 6656:], pos=ints(N), cells=ints(N)):
    qsa.qsa_prep_batched(q, k, v, Z, Z, pos, cells, n, POOL, Z, None, Z, Z, Z, Z)


def refused(fn, *args, **kw):
    with pytest.raises(qsa.QSAError) as e:
        fn(*args, **kw)
    assert e.value.code == qsa.QSA_ERR_INVALID_ARG
    return str(e.value)


def test_rows_with_a_stride(lib):
    wide = torch.zeros(N, 3, 28, 256, dtype=torch.float16)
    for q, k, v, strides in [(FUSED[:, :6144], FUSED[:, 6144:6656], FUSED[:, 6656:], [7168] * 3),
                             (FUSED.view(N, 28, 256)[:, :24], FUSED.view(N, 28, 256)[:, 24:26], FUSED[:, 6656:], [7168] * 3),
                             (wide[:, 0, :24], wide[:, 1, :2], wide[:, 2, 4:6], [21504] * 3),
                             (torch.zeros(N, 24, 256), torch.zeros(N, 2, 256), torch.zeros(N + 3, 512), [6144, 512, 512])]:
        prep(q=q, k=k, v=v)
        assert list(lib["qsa_prep_batched"][3:6]) == strides
    prep(n=1, q=torch.zeros(24, 256), k=torch.zeros(512), v=torch.zeros(1, 2, 256))
    assert list(lib["qsa_prep_batched"][3:6]) == [6144, 512, 512]


@pytest.mark.parametrize("q", [
    torch.zeros(N, 24, 512)[:, :, :256],            # heads apart
    torch.zeros(N, 256, 24).transpose(1, 2),        # dims apart
    torch.zeros(2, N // 2, 24, 256),                # batched: fewer first rows than tokens
    torch.zeros(N, 12, 256),                        # half a row
    torch.zeros(24, N, 256).transpose(0, 1),        # heads first
], ids=["heads", "dims", "batch", "half", "heads first"])
def test_rows_that_do_not_lie_together(lib, q):
    assert "q_raw" in refused(prep, q=q)
    assert not lib


def test_one_row_that_does_not_lie_together(lib):
    assert "q_raw" in refused(prep, n=1, q=torch.zeros(24, 512)[:, :256], pos=ints(1), cells=ints(1))


@pytest.mark.parametrize("pos", [ints(N, 3)[:, :1], ints(3, N).T, ints(N, 1).expand(N, 3), ints(2 * N)[::2], ints(N - 1),
                                 ints(N - 1, 3), ints(N, dtype=torch.int64), torch.zeros(N)],
                         ids=["one axis of three", "axes first", "one position thrice", "every other", "short", "short rows",
                              "int64", "float"])
def test_positions(lib, pos):
    assert "pos" in refused(prep, pos=pos)
    assert not lib


def test_good_positions(lib):
    for pos, axes in ((ints(N), 1), (ints(N, 1), 1), (ints(N, 3), 3), (ints(N + 4), 1), (ints(3, N).T.contiguous(), 3)):
        prep(pos=pos)
        assert lib["qsa_prep_batched"][9] == axes and lib["qsa_prep_batched"][8] == pos.data_ptr()


BAD = [ints(2 * N)[::2], ints(N - 1), ints(N, dtype=torch.int64)]


@pytest.mark.parametrize("bad", BAD, ids=["strided", "short", "int64"])
def test_cells(lib, bad):
    assert "cells" in refused(prep, cells=bad)
    assert "cells" in refused(qsa.qsa_cache_read, Z, Z, Z, Z, POOL, bad, N, Z, Z)
    assert not lib


def tree(seqs=ints(2, 4), masks=ints(N, 2)):
    qsa.qsa_tree_attention(Z, Z, Z, Z, Z, POOL, seqs, 2, N, masks, 50, None, Z)


@pytest.mark.parametrize("bad", [ints(N, 4)[:, :2], ints(2, N).T, ints(N - 1, 2), ints(N, 2, dtype=torch.int64)],
                         ids=["words of a wider mask", "words first", "short", "int64"])
def test_masks(lib, bad):
    assert "tree" in refused(tree, masks=bad)
    assert not lib


@pytest.mark.parametrize("bad", [ints(2, 5)[:, :4], ints(4, 2).T, ints(1, 4), ints(2, 4, dtype=torch.int64)],
                         ids=["wider", "columns first", "short", "int64"])
def test_tables(lib, bad):
    assert "seqs" in refused(tree, seqs=bad)
    assert "seqs" in refused(qsa.qsa_cache_commit, Z, Z, Z, Z, POOL, bad, 2, ints(2, 3), ints(2))
    assert not lib


def test_paths(lib):
    for path, n_path, name in ((ints(2, 8)[:, :3], ints(2), "path"), (ints(1, 3), ints(2), "path"),
                               (ints(2, 3), ints(1), "n_path"), (ints(2, 3), ints(4)[::2], "n_path"),
                               (ints(2, 3, dtype=torch.int64), ints(2), "path")):
        assert name in refused(qsa.qsa_cache_commit, Z, Z, Z, Z, POOL, ints(2, 4), 2, path, n_path)
    assert not lib
    qsa.qsa_cache_commit(Z, Z, Z, Z, POOL, ints(2, 4), 2, ints(2, 3), ints(2))
    assert lib["qsa_cache_commit"][9] == 3


def test_nothing_to_do(lib):
    tree(seqs=ints(2, 4), masks=torch.zeros(N, 2, dtype=torch.int32).view(torch.uint32))
    qsa.qsa_tree_attention(Z, Z, Z, Z, Z, POOL, ints(0, 4), 0, 0, ints(0, 1), 50, None, Z)
    qsa.qsa_cache_commit(Z, Z, Z, Z, POOL, ints(0, 4), 0, ints(0, 3), ints(0))
    qsa.qsa_cache_read(Z, Z, Z, Z, POOL, ints(0), 0, Z, Z)
    prep(n=0, q=FUSED[:0, :6144], k=FUSED[:0, :512], v=FUSED[:0, :512], pos=ints(0), cells=ints(0))
    assert len(lib) == 4


def test_sections_are_whole_numbers_each_time():
    # the parameter blocks are kept by value: an equal float, or a tensor that changes, must not find an earlier one
    good = (10000.0, 256, 1e-6, (32, 48, 48))
    assert list(qsa._rope(good).sections) == [32, 48, 48]
    assert list(qsa._rope((1e4, 256, 1e-6, [32, 48, 48])).sections) == [32, 48, 48]
    with pytest.raises(TypeError):
        qsa._rope((10000.0, 256, 1e-6, (32.0, 48.0, 48.0)))
    sec = [torch.tensor(32), torch.tensor(48), torch.tensor(48)]
    assert list(qsa._rope((1e4, 256, 1e-6, sec)).sections) == [32, 48, 48]
    sec[0].fill_(16)
    sec[1].fill_(64)
    assert list(qsa._rope((1e4, 256, 1e-6, sec)).sections) == [16, 64, 48]
