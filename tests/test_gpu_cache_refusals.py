"""What the binding refuses of CUDA tensors: wrong types, shapes, strides and sizes, before anything is launched; and empty calls."""
import pytest
import torch

from mxfp8_block_scaled_07_b200 import mx

pytestmark = pytest.mark.gpu


@pytest.fixture()
def parts():
    cache = mx.cache_create(4, 2, 64, 16)
    i = dict(dtype=torch.int32, device="cuda")
    return dict(cache=cache, page_table=torch.zeros((3, 2), **i), lengths=torch.ones(3, **i), row_offsets=torch.tensor([0, 1, 2, 3], **i),
                q=torch.zeros((3, 4, 64), dtype=torch.bfloat16, device="cuda"), k=torch.zeros((3, 2, 64), dtype=torch.bfloat16, device="cuda"),
                table=torch.zeros((32, 64), device="cuda"))


def append(p, **kw):
    p = {**p, **kw}
    return mx.cache_append(p["k"], p.get("v", p["k"]), p["cache"], p["page_table"], p["lengths"], p["row_offsets"], q=p["q"], table=p["table"],
                           out=p.get("out"))


def attend(p, **kw):
    p = {**p, **kw}
    return mx.cache_attention(p["q"], p["cache"], p["page_table"], p["lengths"], p["row_offsets"], scale=p.get("scale"), window=p.get("window", 0),
                              return_lse=p.get("return_lse", False), out=p.get("out"))


def test_refusals(parts):
    p = parts
    c = p["cache"]
    common = [dict(page_table=p["page_table"].long()), dict(page_table=p["page_table"][0]), dict(page_table=p["page_table"].cpu()),
              dict(lengths=p["lengths"].long()), dict(lengths=p["lengths"][:2]), dict(row_offsets=p["row_offsets"][:3]),
              dict(row_offsets=p["row_offsets"].long()), dict(row_offsets=p["row_offsets"][::2].repeat(2)[::1][:3]), dict(cache=c[:3]),
              dict(cache=list(c)), dict(cache=(c.k.float(), *c[1:])), dict(cache=(c.k, c.v[:3], *c[2:])), dict(cache=(c.k, c.v, c.k_scale, c.v_scale.cpu())),
              dict(cache=(c.k.transpose(1, 2), c.v.transpose(1, 2), *c[2:])), dict(q=p["q"].half()), dict(q=p["q"].cpu()), dict(q=p["q"][:, :, :32]),
              dict(q=p["q"].transpose(1, 2).contiguous().transpose(1, 2))]
    for kw in common:
        for call in (append, attend):
            with pytest.raises(mx.MxError):
                call(p, **kw)
    two = torch.zeros((2, 4, 64), dtype=torch.bfloat16, device="cuda")
    for kw in (dict(k=p["k"].float()), dict(k=p["k"][:, :1]), dict(v=p["k"][:2]), dict(table=p["table"].double()), dict(table=p["table"][:, :24].contiguous()),
               dict(table=p["table"].cpu()), dict(out=two), dict(q=two), dict(out=p["q"].float()), dict(row_offsets=None, k=p["k"][:2], q=two),
               dict(k=torch.zeros((3, 2, 68), dtype=torch.bfloat16, device="cuda")[:, :, :64])):
        with pytest.raises(mx.MxError):
            append(p, **kw)
    for kw in (dict(q=p["q"][:, :3]), dict(scale=0.0), dict(scale=float("nan")), dict(out=two), dict(out=p["q"].float()), dict(return_lse=True, out=(p["q"],)),
               dict(return_lse=True, out=(p["q"].clone(), torch.zeros((3, 4), dtype=torch.float64, device="cuda"))), dict(row_offsets=None, q=two)):
        with pytest.raises(mx.MxError):
            attend(p, **kw)
    x = torch.zeros((3, 2, 64), device="cuda")
    for args in ((x.double(), p["table"]), (x, p["table"].half()), (x, p["table"][0]), (x, p["table"].cpu()), (x, p["table"][:, :31].contiguous()),
                 (x[:, :, :32], p["table"]), (x[0], p["table"]), (x, p["table"], torch.zeros(2, dtype=torch.int32, device="cuda")),
                 (x, p["table"], torch.zeros(3, device="cuda")), (x, p["table"], None, False, x.half()), (x, p["table"], None, False, x[:2]),
                 (torch.zeros((33, 1, 64), device="cuda"), p["table"])):
        with pytest.raises(mx.MxError):
            mx.rope(*args)
    torch.cuda.synchronize()
    assert mx.device_error() == 0


def test_nothing_to_do(parts):
    p = parts
    i = dict(dtype=torch.int32, device="cuda")
    none = dict(page_table=torch.zeros((0, 2), **i), lengths=torch.zeros(0, **i), row_offsets=None, q=p["q"][:0], k=p["k"][:0])
    assert append(p, **none).shape == (0, 4, 64)
    out, lse = attend(p, **none, return_lse=True)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    assert mx.rope(p["k"][:0], p["table"]).shape == (0, 2, 64) and mx.rope(p["k"][:, :0], p["table"]).shape == (3, 0, 64)
    before = [t.clone() for t in p["cache"]]
    empty = dict(lengths=torch.zeros(3, **i))                     # padding sequences of a captured batch
    assert not append(p, **empty).any() and not attend(p, **empty).any()
    assert not append(p, **empty, row_offsets=None).any() and not attend(p, **empty, row_offsets=None).any()
    assert all(torch.equal(a, b) for a, b in zip(p["cache"], before)) and mx.device_error() == 0


def test_given_outputs(parts):
    p = parts
    out, lse = torch.empty_like(p["q"]), torch.empty((3, 4), device="cuda")
    got = attend(p, return_lse=True, out=(out, lse))
    assert got[0] is out and got[1] is lse
    assert attend(p, out=out) is out and append(p, out=p["q"]) is p["q"]
