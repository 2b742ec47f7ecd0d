"""Host-side refusals of the serving-step calls: status codes before any launch (no GPU needed), and the binding's
checks of types, shapes and devices."""
import ctypes

import pytest
import torch

import compressed_sparse_kv_b200 as K

Z = ctypes.c_void_p(0)
BIG = 1 << 40


def err(rc):
    return rc, K.lib().dsv4kv_last_error().decode()


def table_update(**kw):
    a = dict(t_old=16, t_new=16, batch=2, t_max=1000, window=128, stride=4, lookahead=0, page_rows=64, table=16,
             table_stride=8, pool_pages=10, free=16, cap=10, count=16, out=16, ws=16, ws_bytes=16, stream=Z)
    a.update(kw)
    return err(K.lib().dsv4kv_block_table_update(*a.values()))


@pytest.mark.parametrize("kw,code,text", [
    (dict(batch=-1), 1, "sizes"), (dict(batch=4097), 2, "batch"), (dict(t_max=1 << 30), 2, "t_max"),
    (dict(t_max=-1), 1, "sizes"), (dict(lookahead=129), 1, "lookahead"), (dict(lookahead=-1), 1, "lookahead"),
    (dict(window=70000, lookahead=0), 2, "window"), (dict(t_old=Z), 1, "lengths"), (dict(ws=Z), 3, "workspace"),
    (dict(ws_bytes=8), 3, "workspace"), (dict(ws=24), 3, "workspace"), (dict(stride=-1), 1, "stride"),
    (dict(page_rows=0), 1, "page_rows"), (dict(page_rows=96), 1, "page_rows"), (dict(pool_pages=0), 2, "pool"),
    (dict(pool_pages=1 << 25), 2, "pool"), (dict(table_stride=3), 1, "table_stride"), (dict(table=Z), 1, "table"),
    (dict(cap=-1), 1, "free"), (dict(free=Z), 1, "free"), (dict(count=Z), 1, "free"), (dict(out=Z), 1, "free"),
    (dict(batch=4096, t_max=(1 << 30) - 1, stride=1, table_stride=1 << 25), 2, "pages"),
])
def test_block_table_update(kw, code, text):
    rc, msg = table_update(**kw)
    assert rc == code and text in msg, (rc, msg)


def slots(**kw):
    pt = lambda **k: ctypes.byref(K.PageTableDesc(**{**dict(table=16, page_rows=64, table_stride=8, pool_pages=10), **k}))  # noqa: E731
    a = dict(t_old=16, t_new=16, batch=2, t_max=1000, window=128, stride=4, lookahead=0, comp=pt(), win=pt(), capacity=64,
             cu=16, seq=16, pos=16, win_slot=16, comp_slot=16, ws=16, ws_bytes=16, stream=Z)
    a.update({k: (pt(**v) if isinstance(v, dict) else v) for k, v in kw.items()})
    return err(K.lib().dsv4kv_slot_map(*a.values()))


@pytest.mark.parametrize("kw,code,text", [
    (dict(stride=0), 1, "stride"), (dict(capacity=-1), 1, "capacity"), (dict(capacity=1 << 31), 2, "capacity"),
    (dict(cu=Z), 1, "output"), (dict(seq=8), 1, "output"), (dict(win=None), 1, "window table"),
    (dict(win=dict(table_stride=1)), 1, "table_stride"), (dict(comp=dict(page_rows=32)), 1, "page_rows"),
    (dict(comp=dict(table=None)), 1, "table"), (dict(lookahead=200), 1, "lookahead"), (dict(batch=5000), 2, "batch"),
])
def test_slot_map(kw, code, text):
    rc, msg = slots(**kw)
    assert rc == code and text in msg, (rc, msg)


def paged(**k):
    return ctypes.byref(K.PagedDesc(**{**dict(fmt=0, dim=512, page_rows=64, table_stride=16, pool_pages=10, table=16,
                                              codes=16, scales=None), **k}))


def append(**kw):
    a = dict(s_new=16, w=16, batch=2, capacity=8, cu=16, seq=16, pos=16, win_slot=16, comp_slot=16, k_taps=8, stride=4,
             window=128, lookahead=0, max_new=8, rope_dim=64, base=1e4, ring=16, win=paged(), comp=paged(), ws=16,
             ws_bytes=16, stream=Z)
    a.update({k: (paged(**v) if isinstance(v, dict) else v) for k, v in kw.items()})
    return err(K.lib().dsv4kv_append_paged(*a.values()))


@pytest.mark.parametrize("kw,code,text", [
    (dict(stride=0), 1, "sizes"), (dict(k_taps=0), 1, "sizes"), (dict(max_new=-1), 1, "sizes"),
    (dict(lookahead=129), 1, "lookahead"), (dict(rope_dim=63), 1, "rope_dim"), (dict(rope_dim=514), 1, "rope_dim"),
    (dict(base=0.0), 1, "rope_base"), (dict(ws=Z), 3, "workspace"), (dict(s_new=8), 1, "misaligned"),
    (dict(ring=Z), 1, "null"), (dict(cu=Z), 1, "slot map"), (dict(win=None), 1, "descriptor"),
    (dict(comp=None), 1, "descriptor"), (dict(comp=dict(fmt=7)), 2, "format"), (dict(comp=dict(dim=256)), 2, "dim"),
    (dict(comp=dict(fmt=1)), 1, "scales"), (dict(comp=dict(fmt=1, scales=16)), 2, "format"),
    (dict(comp=dict(codes=None)), 1, "codes"), (dict(comp=dict(pool_pages=0)), 2, "pool"),
    (dict(comp=dict(fmt=3, scales=16), win=dict(fmt=3, scales=16), rope_dim=32), 2, "rope_dim"),
    (dict(capacity=1 << 31), 2, "large"),
])
def test_append_paged(kw, code, text):
    rc, msg = append(**kw)
    assert rc == code and text in msg, (rc, msg)


def test_append_of_nothing_is_ok():
    assert append(capacity=0, s_new=Z)[0] == 0 and append(batch=0, s_new=Z)[0] == 0


def tree(**kw):
    draft = lambda **k: ctypes.byref(K.CacheDesc(**{**dict(fmt=0, dim=512, rows=20, codes=16, scales=None), **k}))  # noqa: E731
    a = dict(q=16, comp=paged(), win=paged(), draft=draft(), cu=16, parent=16, idx=Z, batch=2, heads=64, nodes=20,
             max_nodes=10, t_seq=16, t_max=1000, window=128, stride=4, k=0, scale=0.04, rope_dim=64, base=1e4, fp32=0,
             out=16, ws=16, ws_bytes=BIG, stream=Z)
    a.update({k: ((draft if k == "draft" else paged)(**v) if isinstance(v, dict) else v) for k, v in kw.items()})
    return err(K.lib().dsv4kv_tree_decode_paged(*a.values()))


@pytest.mark.parametrize("kw,code,text", [
    (dict(batch=0), 1, "batch"), (dict(batch=1025), 2, "batch"), (dict(t_seq=Z), 1, "t_seq"), (dict(stride=0), 1, "sizes"),
    (dict(nodes=-1), 1, "sizes"), (dict(max_nodes=0), 1, "sizes"), (dict(max_nodes=257), 2, "max_nodes"),
    (dict(heads=0), 2, "heads"), (dict(heads=129), 2, "heads"), (dict(t_max=1 << 30), 2, "t_max"),
    (dict(idx=16, k=0), 2, "k must"), (dict(idx=16, k=2049), 2, "k must"), (dict(rope_dim=514), 1, "rope_dim"),
    (dict(base=-1.0), 1, "rope_base"), (dict(cu=Z), 1, "cu"), (dict(comp=dict(table_stride=2)), 1, "table_stride"),
    (dict(comp=dict(dim=128)), 2, "dim"), (dict(comp=dict(table=None)), 1, "table"), (dict(win=dict(codes=8)), 1, "codes"),
    (dict(win=dict(table_stride=1)), 1, "table_stride"), (dict(draft=dict(rows=19)), 1, "rows"),
    (dict(draft=dict(fmt=2, scales=16)), 2, "format"), (dict(comp=dict(fmt=1, scales=16)), 2, "format"),
    (dict(comp=dict(fmt=3, scales=16), win=dict(fmt=3, scales=16), draft=dict(fmt=3, scales=16), rope_dim=32), 2, "rope_dim"),
    (dict(ws=Z), 3, "workspace"), (dict(ws=8), 3, "workspace"), (dict(ws_bytes=1000), 3, "workspace"),
    (dict(q=8), 1, "q/out"), (dict(out=Z), 1, "q/out"), (dict(parent=Z), 1, "parent"),
    (dict(t_max=100, comp=dict(table=None, codes=None), window=64, stride=4), 1, "table"),
    (dict(t_max=60, max_nodes=10, window=64, comp=dict(codes=None)), 1, "codes"),   # entries within reach of a draft only
])
def test_tree_decode_paged(kw, code, text):
    rc, msg = tree(**kw)
    assert rc == code and text in msg, (rc, msg)


def test_tree_of_no_nodes_is_ok_and_sizes():
    assert tree(nodes=0, q=Z, out=Z)[0] == 0
    assert K.tree_decode_paged_workspace_bytes(1, 64, 1, 1, 100) > 0
    assert K.tree_decode_paged_workspace_bytes(1, 300, 1, 1, 100) == 0
    assert K.paged_step_workspace_bytes(8) == 16 and K.paged_step_workspace_bytes(-1) == 0


def test_the_binding_refuses_what_it_cannot_marshal():
    i64 = torch.zeros(2, dtype=torch.int64)
    i32 = torch.zeros(2, dtype=torch.int32)
    pt = K.PageTable(torch.zeros(2, 4, dtype=torch.int32), 64, 4)
    count = torch.zeros(1, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA device"):
        K.block_table_update(i64, i64, pt, i32, count, 100)
    with pytest.raises(ValueError, match="t_new"):
        K.block_table_update(i64, torch.zeros(3, dtype=torch.int64), pt, i32, count, 100)
    with pytest.raises(ValueError, match="t_old"):
        K.block_table_update(i32, i64, pt, i32, count, 100)
    with pytest.raises(ValueError, match="table"):
        K.slot_map(i64, i64, K.PageTable(torch.zeros(4, 2, dtype=torch.int32).T, 64, 4), pt, 8, 100)
    m = K.new_slot_map(2, 8, device="cpu")
    x, w, ring = torch.zeros(8, 512, dtype=torch.bfloat16), torch.zeros(8, 512), torch.zeros(2, 136, 512, dtype=torch.bfloat16)
    c = K.PagedCache(0, torch.zeros(128, 512, dtype=torch.bfloat16), torch.zeros(2, 4, dtype=torch.int32), 64)
    with pytest.raises(ValueError, match="s_new"):
        K.append_paged(x[:7], w, m, ring, c, c, 4)
    with pytest.raises(ValueError, match="s_new"):
        K.append_paged(torch.zeros(8, 1024, dtype=torch.bfloat16)[:, ::2], w, m, ring, c, c, 4)
    with pytest.raises(ValueError, match="raw_ring"):
        K.append_paged(x, w, m, ring[:, :130], c, c, 4)
    with pytest.raises(ValueError, match="comp.codes"):
        K.append_paged(x, w, m, ring, c, K.PagedCache(1, torch.zeros(128, 256, dtype=torch.uint8), c.table, 64,
                                                      torch.zeros(128)), 4)
    q, cu = torch.zeros(3, 4, 512, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    d = K.Cache(0, torch.zeros(1, 2, 512, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="draft"):
        K.tree_decode_paged(q, c, c, d, cu, torch.zeros(3, dtype=torch.int32), i64, 100, 4)
    with pytest.raises(ValueError, match="parent"):
        K.tree_decode_paged(q, c, c, d, cu, torch.zeros(3, dtype=torch.int64), i64, 100, 4)
    with pytest.raises(ValueError, match="q must"):
        K.tree_decode_paged(q.float(), c, c, d, cu, torch.zeros(3, dtype=torch.int32), i64, 100, 4)


@pytest.mark.parametrize("fmt,codes,scales,text", [
    (0, torch.float32, None, "comp.codes"), (0, torch.float16, None, "comp.codes"), (0, torch.uint8, None, "comp.codes"),
    (1, torch.bfloat16, torch.float32, "comp.codes"), (1, torch.uint8, torch.float64, "comp.scales"),
    (1, torch.uint8, torch.bfloat16, "comp.scales"), (1, torch.uint8, torch.int32, "comp.scales"),
    (2, torch.int32, torch.uint8, "comp.codes"), (2, torch.uint8, torch.float32, "comp.scales"),
    (3, torch.float16, torch.float32, "comp.codes"), (3, torch.uint8, torch.float16, "comp.scales"),
])
def test_the_binding_refuses_rows_of_another_type(fmt, codes, scales, text):
    """Tensors with room for the rows, whose bytes would be taken for something else."""
    m = K.new_slot_map(2, 8, device="cpu")
    x, w, ring = torch.zeros(8, 512, dtype=torch.bfloat16), torch.zeros(8, 512), torch.zeros(2, 136, 512, dtype=torch.bfloat16)
    c = K.PagedCache(fmt, torch.zeros(128, 1024, dtype=codes), torch.zeros(2, 4, dtype=torch.int32), 64,
                     None if scales is None else torch.zeros(128, 64, dtype=scales))
    with pytest.raises(ValueError, match=text + " must be (bf16|bytes|float32)"):
        K.append_paged(x, w, m, ring, c, c, 4)
    i64, i32 = torch.zeros(2, dtype=torch.int64), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match=text):
        K.tree_decode_paged(torch.zeros(3, 4, 512, dtype=torch.bfloat16), c, c, K.Cache(fmt, c.codes[None]), i32, i32, i64,
                            100, 4)


@pytest.mark.parametrize("fmt,codes,scales", [
    (0, torch.bfloat16, None), (0, torch.uint16, None), (0, torch.int16, None), (1, torch.uint8, torch.float32),
    (1, torch.float8_e4m3fn, torch.float32), (2, torch.int8, torch.float8_e4m3fn), (3, torch.uint8, torch.float32),
])
def test_the_binding_takes_every_spelling_of_a_format(fmt, codes, scales):
    c = K.PagedCache(fmt, torch.zeros(128, 1024, dtype=codes), torch.zeros(2, 4, dtype=torch.int32), 64,
                     None if scales is None else torch.zeros(128, 64, dtype=scales))
    m = K.new_slot_map(2, 8, device="cpu")
    with pytest.raises(ValueError, match="CUDA device"):        # the last check, behind those of the rows
        K.append_paged(torch.zeros(8, 512, dtype=torch.bfloat16), torch.zeros(8, 512), m,
                       torch.zeros(2, 136, 512, dtype=torch.bfloat16), c, c, 4)
