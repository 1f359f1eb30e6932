"""Sort tiles of both sizes (1024 keys up to 2^19 keys, 4096 beyond and for one
tile): the sorted positions and their runs against numpy's stable sort at the
edges, and a workspace that a shorter batch never outgrows."""
import ctypes as C

import numpy as np
import pytest
import torch

eb = pytest.importorskip("recommender_embedding_tables_amd.embtab",
                         reason="libembtab.so not built")

EDGE = 1 << 19


def test_a_longer_batch_never_needs_less_workspace():
    d = eb.emb_table_desc_t()
    rows = (C.c_int64 * 2)(1000, 24)
    d.num_tables, d.dim, d.rows_per_table = 2, 4, C.cast(rows, C.c_void_p)
    d.weights, d.accum, d.state = 0x10000000, 0x20000000, 0x30000000
    d.max_load, d.init_storage = 0.625, 0
    st, h = eb.emb_table_create(d, 0)
    assert st == eb.EMB_OK
    sizes = [0, 1, 1023, 1024, 4095, 4096, 4097, 5000, 8192, 100_000, EDGE - 4096, EDGE - 1, EDGE,
             EDGE + 1, EDGE + 4096, 5_000_000]
    got = [eb.emb_workspace_bytes(h, 64, n) for n in sizes]
    eb.emb_table_destroy(h)
    assert all(a <= b for a, b in zip(got, got[1:])), list(zip(sizes, got))


@pytest.mark.gpu
@pytest.mark.parametrize("n", [4096, 4097, 5121, 300_001, EDGE, EDGE + 1, (1 << 22) + 1])
@pytest.mark.parametrize("rows", [[700, 90], [200_000, 3, 1_500_000]])
def test_sorted_positions(n, rows):
    dev = torch.device("cuda")
    r = np.random.default_rng(n + len(rows))
    B, T = 97, len(rows)
    cut = np.sort(r.integers(0, n + 1, B * T - 1))
    offsets = np.concatenate([[0], cut, [n]]).astype(np.int64)
    table = np.repeat(np.arange(B * T) // B, np.diff(offsets))
    ids = (r.random(n) ** 2 * np.array(rows)[table]).astype(np.int64)
    key = ids + np.concatenate([[0], np.cumsum(rows)])[table]
    tabs = eb.EmbTables(rows, 4)
    out = {k: torch.empty(n + 1, dtype=torch.int32, device=dev)
           for k in ("sorted", "perm", "unique", "counts", "seg_off", "inverse")}
    num = torch.zeros(1, dtype=torch.int32, device=dev)
    ws, need = tabs.workspace(B, n)
    ws.fill_(255)
    eb.check(eb.emb_debug_sort_unique(
        tabs.handle, torch.from_numpy(offsets).to(dev), torch.from_numpy(ids).to(dev), B, n,
        out["sorted"], out["perm"], out["unique"], out["counts"], out["seg_off"], out["inverse"],
        num, ws, need), "sort_unique")
    torch.cuda.synchronize()
    assert eb.emb_status_sync(tabs.handle)[0] == eb.EMB_OK
    perm = np.argsort(key, kind="stable")
    uniq, first, inverse, counts = np.unique(key, return_index=True, return_inverse=True,
                                             return_counts=True)
    u = uniq.size
    assert int(num) == u
    got = {k: v.cpu().numpy() for k, v in out.items()}
    assert np.array_equal(got["perm"][:n], perm)
    assert np.array_equal(got["sorted"][:n], key[perm])
    assert np.array_equal(got["unique"][:u], uniq)
    assert np.array_equal(got["counts"][:u], counts)
    assert np.array_equal(got["inverse"][:n], inverse)
    assert np.array_equal(got["seg_off"][:u + 1], np.concatenate([[0], np.cumsum(counts)]))
    tabs.close()
