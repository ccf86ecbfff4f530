"""CPU-only checks of the layer operators' C ABI: the header is strict C99, the
binding's structures have the C ones' layout, and bad arguments are refused on
the host before any CUDA call (the addresses here are never dereferenced)."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID = 1


@pytest.fixture(scope="module")
def ep():
    from combine_get_dispatch_layout_gb300.build import build
    import combine_get_dispatch_layout_gb300 as ep

    build()
    ep.lib()
    return ep


STRUCTS = {"ep_router_config_t": "RouterConfig", "ep_cache_t": "Cache", "ep_append_config_t": "AppendConfig",
           "ep_attention_config_t": "AttentionConfig", "ep_w4_config_t": "W4Config"}


def test_structures_match_the_header(ep, tmp_path):
    lines = []
    for c, py in STRUCTS.items():
        lines.append(f'printf("{c} %zu\\n", sizeof({c}));')
        for field, _ in getattr(ep.layer, py)._fields_:
            lines.append(f'printf("{c}.{field} %zu\\n", offsetof({c}, {field}));')
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include "ep_layer.h"\nint main(void) {\n' + "\n".join(lines) + "\nreturn 0;\n}\n")
    exe = str(tmp_path / "s")
    subprocess.run(["gcc", "-std=c99", "-pedantic", "-Wall", "-Wextra", "-Werror", "-I",
                    os.path.join(ROOT, "include"), str(src), "-o", exe], check=True)
    got = dict(x.split() for x in subprocess.run([exe], check=True, capture_output=True, text=True).stdout.splitlines())
    for c, py in STRUCTS.items():
        s = getattr(ep.layer, py)
        assert int(got.pop(c)) == ctypes.sizeof(s)
        for field, _ in s._fields_:
            assert int(got.pop(f"{c}.{field}")) == getattr(s, field).offset, (c, field)
    assert not got


def router(ep, **kw):
    a = dict(logits=16, ld=8, bias=None, T=4, E=8, K=2, idx=16, w=16, dtype=ep.EP_DTYPE_FP32, score=0, scale=1.0,
             groups=1, keep=1, top=1, cfg=True)
    a.update(kw)
    cfg = ep.layer.RouterConfig(a["dtype"], a["score"], 1, a["scale"], a["groups"], a["keep"], a["top"])
    L = ep.lib()
    return (L.ep_router_topk(a["logits"], a["ld"], a["bias"], a["T"], a["E"], a["K"], cfg if a["cfg"] else None,
                             a["idx"], a["w"], None),
            L.ep_router_topk_backward(a["logits"], a["ld"], a["idx"], 2, a["w"], a["T"], a["E"], a["K"],
                                      cfg if a["cfg"] else None, a["logits"], a["ld"], None))


@pytest.mark.parametrize("kw", [dict(logits=None), dict(logits=18), dict(ld=7), dict(T=-1), dict(E=0, ld=0),
                                dict(E=4097, ld=4097), dict(K=0), dict(K=33), dict(idx=None), dict(idx=12),
                                dict(w=None), dict(w=18), dict(dtype=1), dict(dtype=5), dict(score=2),
                                dict(scale=float("nan")), dict(cfg=False)])
def test_router_rejects(ep, kw):
    assert router(ep, **kw) == (INVALID, INVALID)


@pytest.mark.parametrize("kw", [dict(bias=18), dict(groups=3), dict(groups=-1), dict(groups=64, E=128, ld=128),
                                dict(groups=4, keep=0), dict(groups=4, keep=5), dict(top=3), dict(top=-1)])
def test_router_rejects_groups_and_bias(ep, kw):
    assert router(ep, **kw)[0] == INVALID


def test_router_backward_rejects_short_index_rows(ep):
    cfg = ep.layer.RouterConfig(ep.EP_DTYPE_FP32, 0, 1, 1.0, 1, 1, 1)
    assert ep.lib().ep_router_topk_backward(16, 8, 16, 1, 16, 4, 8, 2, cfg, 16, 8, None) == INVALID


def test_empty_router_needs_nothing(ep):
    assert router(ep, T=0, logits=None, idx=None, w=None) == (0, 0)


def cache_struct(ep, **kw):
    a = dict(dtype=0, page=16, pages=4, kp=2048, ks=128, kh=64, vp=2048, vs=128, vh=64, k_scale=1.0, v_scale=1.0)
    a.update(kw)
    return ep.layer.Cache(a["dtype"], a["page"], a["pages"], a["kp"], a["ks"], a["kh"], a["vp"], a["vs"], a["vh"],
                          a["k_scale"], a["v_scale"])


BAD_CACHES = [dict(dtype=2), dict(dtype=3), dict(dtype=4), dict(page=0), dict(pages=-1), dict(pages=1 << 33),
              dict(page=1 << 20, pages=1 << 21), dict(kp=2052), dict(vh=63), dict(ks=-8), dict(dtype=1, kh=72),
              dict(dtype=1, k_scale=0.0), dict(dtype=1, v_scale=float("inf")), dict(dtype=1, v_scale=float("nan"))]


def append(ep, cache=None, **kw):
    a = dict(q=16, k=16, v=16, pos=16, slots=16, cs=16, T=4, q_out=16, kc=16, vc=16, err=None, dtype=0, h=4, n=2, d=64,
             rot=64, q_ld=256, k_ld=128, v_ld=128, qo_ld=256, most=9, cfg=True)
    a.update(kw)
    cfg = ep.layer.AppendConfig(a["dtype"], a["h"], a["n"], a["d"], a["rot"], 0, a["q_ld"], a["k_ld"], a["v_ld"],
                                a["qo_ld"], a["most"])
    return ep.lib().ep_kv_append(a["q"], a["k"], a["v"], a["pos"], a["slots"], a["cs"], a["T"],
                                 cfg if a["cfg"] else None, a["q_out"], a["kc"], a["vc"],
                                 cache if cache is not None else cache_struct(ep), a["err"], None)


@pytest.mark.parametrize("kw", [dict(q=None), dict(q=24), dict(k=None), dict(v=24), dict(pos=None), dict(pos=20),
                                dict(slots=None), dict(slots=20), dict(cs=None), dict(cs=18), dict(T=-1),
                                dict(q_out=None), dict(kc=None), dict(vc=24), dict(err=18), dict(dtype=1), dict(dtype=4),
                                dict(h=-1), dict(n=0), dict(d=60), dict(d=0), dict(d=2048), dict(rot=63), dict(rot=66),
                                dict(rot=-2), dict(q_ld=255), dict(q_ld=260), dict(k_ld=120), dict(v_ld=132),
                                dict(qo_ld=248), dict(most=0), dict(cfg=False)])
def test_append_rejects(ep, kw):
    assert append(ep, **kw) == INVALID


@pytest.mark.parametrize("kw", BAD_CACHES)
def test_append_and_attention_reject_caches(ep, kw):
    assert append(ep, cache_struct(ep, **kw)) == INVALID
    assert attention(ep, cache_struct(ep, **kw)) == INVALID


def attention(ep, cache=None, **kw):
    a = dict(q=16, kc=16, vc=16, table=16, lens=16, B=2, out=16, lse=None, work=16, size=1 << 40, dtype=0, h=4, n=2,
             d=64, pages=3, q_ld=256, out_ld=256, table_ld=3, scale=0.1, window=0, cfg=True)
    a.update(kw)
    cfg = ep.layer.AttentionConfig(a["dtype"], a["h"], a["n"], a["d"], a["pages"], a["q_ld"], a["out_ld"],
                                   a["table_ld"], a["scale"], a["window"])
    return ep.lib().ep_paged_attention(a["q"], a["kc"], a["vc"], cache if cache is not None else cache_struct(ep),
                                       a["table"], a["lens"], a["B"], cfg if a["cfg"] else None, a["out"], a["lse"],
                                       a["work"], a["size"], None)


@pytest.mark.parametrize("kw", [dict(q=None), dict(q=24), dict(kc=None), dict(vc=24), dict(table=None), dict(table=18),
                                dict(lens=None), dict(lens=18), dict(B=-1), dict(B=1 << 29, h=4), dict(out=None),
                                dict(out=24), dict(lse=18), dict(work=24), dict(dtype=1), dict(dtype=4), dict(h=3),
                                dict(h=0), dict(n=0), dict(d=60), dict(d=264, q_ld=2048, out_ld=2048), dict(pages=-1),
                                dict(pages=1 << 28, table_ld=1 << 28), dict(q_ld=248), dict(q_ld=260),
                                dict(out_ld=255), dict(table_ld=2), dict(scale=float("inf")), dict(window=-1),
                                dict(cfg=False)])
def test_attention_rejects(ep, kw):
    assert attention(ep, **kw) == INVALID


def test_attention_workspace_rejects(ep):
    for args in [(-1, 4, 2, 64), (2, 0, 2, 64), (2, 4, 0, 64), (2, 4, 3, 64), (2, 4, 2, 0), (2, 4, 2, 60),
                 (2, 4, 2, 264), (1 << 30, 4, 2, 64)]:
        assert ep.lib().ep_paged_attention_workspace(*args) == -1


def experts(ep, **kw):
    a = dict(x=16, rows=4, I=128, w=16, s=16, z=None, off=16, cnt=None, E=2, O=10, y=16, dtype=0, group=64, act=0,
             x_ld=128, y_ld=10, cfg=True, work=16, size=1 << 40)
    a.update(kw)
    cfg = ep.layer.W4Config(a["dtype"], a["group"], a["act"], a["x_ld"], a["y_ld"])
    return ep.lib().ep_expert_w4(a["x"], a["rows"], a["I"], a["w"], a["s"], a["z"], a["off"], a["cnt"], a["E"], a["O"],
                                 cfg if a["cfg"] else None, a["y"], a["work"], a["size"], None)


@pytest.mark.parametrize("kw", [dict(x=None), dict(x=24), dict(rows=-1), dict(rows=1 << 31), dict(I=0), dict(I=96),
                                dict(w=None), dict(w=24), dict(s=None), dict(s=17), dict(off=None), dict(off=18),
                                dict(cnt=18), dict(off=None, E=1, cnt=16), dict(E=0), dict(E=4097), dict(O=0), dict(y=None),
                                dict(y=17), dict(dtype=1), dict(dtype=4), dict(group=16), dict(group=256, I=256, x_ld=256),
                                dict(group=48, I=96, x_ld=96), dict(act=2), dict(act=1, O=9), dict(x_ld=120),
                                dict(x_ld=132), dict(y_ld=9), dict(cfg=False), dict(work=None), dict(work=24), dict(size=100)])
def test_experts_reject(ep, kw):
    assert experts(ep, **kw) == INVALID


def test_experts_workspace_rejects(ep):
    for args in [(-1, 128, 64, 0), (1 << 31, 128, 64, 0), (4, 96, 64, 0), (4, 0, 64, 0), (4, 128, 16, 0), (4, 128, 64, 1)]:
        assert ep.lib().ep_expert_w4_workspace(*args) == -1


def test_empty_calls_need_nothing(ep):
    assert attention(ep, B=0, q=None, out=None, lens=None, table=None) == 0
    assert append(ep, T=0, q=None, k=None, v=None, pos=None, slots=None, cs=None, q_out=None) == 0
    assert experts(ep, rows=0, x=None, w=None, s=None, y=None) == 0


def test_dispatch_still_refuses_the_new_types(ep):
    h = ctypes.c_void_p(None)
    assert (ep.EP_DTYPE_BF16, ep.EP_DTYPE_FP8_E4M3, ep.EP_DTYPE_FP8_E5M2, ep.EP_DTYPE_FP16, ep.EP_DTYPE_FP32) == tuple(range(5))
    assert ep.lib().ep_dispatch(h, 16, 128, ep.EP_DTYPE_FP16, None, 16, None, None, None, 10, None) == INVALID
