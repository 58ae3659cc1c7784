"""Host-side checks of the paged cache and of attention over it (no GPU): the
index arithmetic against plain definitions, and every refusal's status before
anything is enqueued."""
import ctypes as ct
import os
import subprocess

import pytest
import torch

import block_scaled_fp4_amax_amd as fq

HERE = os.path.dirname(os.path.abspath(__file__))
FAKE, MIS = 0x10000, 0x10004
no_gpu = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="placeholder device pointers: host-only validation")


def test_index_arithmetic(tmp_path):
    exe = str(tmp_path / "kv_index_check")
    subprocess.run(["g++", "-O1", "-D_GLIBCXX_ASSERTIONS", "-std=c++17", "-o", exe,
                    os.path.join(HERE, "pins", "kv_index_check.cpp")], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


def cache(**kw):
    d = dict(k_codes=FAKE, k_scales=FAKE, v_codes=FAKE, v_scales=FAKE, k_outer=None, v_outer=None, num_pages=4,
             page_size=16, kv_heads=2, head_dim=64, reserved=0)
    d.update(kw)
    return fq._KvCache(**d)


def status(st):
    assert st != fq.ERR_HIP, "a call reached a launch"
    return st


def append(c=None, cfg=None, tokens=3, k=FAKE, ld_k=128, v=FAKE, ld_v=128, slots=FAKE):
    cfg = cfg if cfg is not None else fq.make_cfg()
    return status(fq.lib().fp4_kv_append(ct.byref(cfg), ct.byref(c if c is not None else cache()), k, ld_k, v, ld_v,
                                         slots, tokens, None))


def read(c=None, cfg=None, tokens=3, k=FAKE, v=FAKE, slots=FAKE):
    cfg = cfg if cfg is not None else fq.make_cfg()
    return status(fq.lib().fp4_kv_read(ct.byref(cfg), ct.byref(c if c is not None else cache()), slots, tokens, k, v,
                                       None))


def args(**kw):
    d = dict(q=FAKE, ld_q=256, page_table=FAKE, kv_lens=FAKE, q_starts=FAKE, sinks=None, out=FAKE, lse=None, scale=0.125,
             batch=2, total_q=5, q_heads=4, table_cols=4, max_q=3, max_kv=64, causal=1, window=0)
    d.update(kw)
    return fq._Attn(**d)


def attn(c=None, cfg=None, ws=None, wsb=0, **kw):
    cfg = cfg if cfg is not None else fq.make_cfg()
    return status(fq.lib().fp4_attn(ct.byref(cfg), ct.byref(c if c is not None else cache()), ct.byref(args(**kw)), ws,
                                    wsb, None))


@no_gpu
@pytest.mark.parametrize("call", [append, read, attn])
def test_cache_rules(call):
    C = fq.make_cfg
    assert call(cfg=C(rounding="stochastic")) == fq.ERR_UNSUPPORTED
    assert call(cfg=C(two_level="outer_block", outer_block_size=64)) == fq.ERR_UNSUPPORTED
    assert call(cfg=C(inner_2d=True)) == fq.ERR_MODE
    assert call(cfg=C(two_level="tensorwise")) == fq.ERR_MODE          # a cache's scale is given
    assert call(cfg=C(two_level="tensorwise", outer_mode=1)) == fq.ERR_NULL
    assert call(cfg=C(two_level="tensorwise", outer_mode=1), c=cache(k_outer=FAKE)) == fq.ERR_NULL
    assert call(cfg=C(two_level="tensorwise", outer_mode=1), c=cache(k_outer=FAKE, v_outer=FAKE + 2)) == fq.ERR_ALIGN
    assert call(cfg=C(format="mxfp4", two_level="tensorwise", outer_mode=1)) == fq.ERR_MODE
    assert call(cfg=C(input_dtype="fp16")) == fq.ERR_DTYPE
    assert call(cfg=C(output_dtype="fp16")) == fq.ERR_DTYPE
    bad = C()
    bad.abi_version = 1
    assert call(cfg=bad) == fq.ERR_ABI
    for kw in (dict(num_pages=-1), dict(kv_heads=0), dict(page_size=0), dict(page_size=8), dict(page_size=40)):
        assert call(c=cache(**kw)) == fq.ERR_SHAPE, kw
    for kw in (dict(head_dim=96), dict(head_dim=0), dict(head_dim=512), dict(page_size=8192), dict(kv_heads=65536),
               dict(num_pages=1 << 31)):
        assert call(c=cache(**kw)) == fq.ERR_UNSUPPORTED, kw
    for n in ("k_codes", "k_scales", "v_codes", "v_scales"):
        assert call(c=cache(**{n: None})) == fq.ERR_NULL
        assert call(c=cache(**{n: MIS})) == fq.ERR_ALIGN


@no_gpu
def test_append_and_read_rules():
    assert append(tokens=-1) == fq.ERR_SHAPE and read(tokens=-1) == fq.ERR_SHAPE
    assert append(ld_k=120) == fq.ERR_SHAPE and append(ld_v=120) == fq.ERR_SHAPE
    assert append(ld_k=132) == fq.ERR_ALIGN
    assert append(cfg=fq.make_cfg(input_dtype="fp32"), ld_k=130) == fq.ERR_ALIGN
    assert append(tokens=(1 << 27) + 1) == fq.ERR_UNSUPPORTED and read(tokens=(1 << 27) + 1) == fq.ERR_UNSUPPORTED
    assert append(ld_k=1 << 32) == fq.ERR_UNSUPPORTED
    assert read(c=cache(kv_heads=64), tokens=1 << 26) == fq.ERR_UNSUPPORTED
    for n in ("k", "v", "slots"):
        assert append(**{n: None}) == fq.ERR_NULL and read(**{n: None}) == fq.ERR_NULL
        assert append(**{n: MIS}) == fq.ERR_ALIGN and read(**{n: MIS}) == fq.ERR_ALIGN
    assert append(tokens=0, k=None, v=None, slots=None) == fq.OK
    assert read(tokens=0, k=None, v=None, slots=None) == fq.OK
    assert append(c=cache(num_pages=0, k_codes=None, k_scales=None, v_codes=None, v_scales=None)) == fq.OK


@no_gpu
def test_attention_rules():
    for kw in (dict(batch=-1), dict(total_q=-1), dict(table_cols=-1), dict(max_q=-1), dict(max_kv=-1), dict(window=-1),
               dict(q_heads=0), dict(q_heads=3), dict(ld_q=248), dict(q_starts=None)):
        assert attn(**kw) == fq.ERR_SHAPE, kw
    for kw in (dict(causal=2), dict(causal=0, window=5), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
               dict(scale=float("inf"))):
        assert attn(**kw) == fq.ERR_MODE, kw
    for kw in (dict(max_kv=(1 << 27) + 1), dict(table_cols=1 << 27), dict(batch=65536), dict(max_q=1 << 22),
               dict(total_q=1 << 30)):
        assert attn(**kw) == fq.ERR_UNSUPPORTED, kw
    assert attn(c=cache(kv_heads=4096), q_heads=4096, batch=4096, ld_q=1 << 20) == fq.ERR_UNSUPPORTED
    for n in ("q", "kv_lens", "out", "page_table"):
        assert attn(**{n: None}) == fq.ERR_NULL
    for n in ("q", "out"):
        assert attn(**{n: MIS}) == fq.ERR_ALIGN
    for n in ("kv_lens", "page_table", "q_starts", "sinks", "lse"):
        assert attn(**{n: FAKE + 2}) == fq.ERR_ALIGN
    assert attn(ld_q=260) == fq.ERR_ALIGN
    for kw in (dict(batch=0, q_starts=FAKE), dict(total_q=0), dict(max_q=0)):
        assert attn(q=None, out=None, **kw) == fq.OK
    long = dict(max_kv=1 << 20, table_cols=1 << 16)
    need = fq.lib().fp4q_attn_workspace_bytes(ct.byref(fq.make_cfg()), ct.byref(cache()), ct.byref(args(**long)))
    assert need > 0
    assert attn(**long) == fq.ERR_WORKSPACE
    assert attn(ws=FAKE, wsb=need - 1, **long) == fq.ERR_WORKSPACE
    assert attn(ws=MIS, wsb=need, **long) == fq.ERR_ALIGN
    assert fq.lib().fp4q_attn_workspace_bytes(ct.byref(fq.make_cfg()), ct.byref(cache()), ct.byref(args(batch=-1))) == 0


@no_gpu
def test_attention_workspace_at_the_ends():
    """Scratch is bounded by what the chip holds, and a call whose units or rows would pass the
    counters does without it."""
    def need(c=None, **kw):
        return fq.lib().fp4q_attn_workspace_bytes(ct.byref(fq.make_cfg()), ct.byref(c if c is not None else cache()),
                                                  ct.byref(args(**kw)))
    one = dict(max_q=1, q_starts=FAKE)
    assert need(max_kv=512, table_cols=32, **one) == 0
    assert need(max_kv=8192, table_cols=512, batch=1024, total_q=1024, **one) == 0       # heads fill the chip
    for n in (1, 7, 64, 500):
        assert 0 < need(max_kv=1 << 27, table_cols=1 << 23, batch=n, total_q=n, **one) < 1 << 28
    # 1000 sequences of 2^27 keys: 2^31 units
    assert need(max_kv=1 << 27, table_cols=1 << 23, batch=1000, total_q=1000, **one) == 0
    # rows of many, split: scratch follows the tensor, until one launch cannot join it
    many = dict(max_q=64, batch=1, max_kv=1 << 20, table_cols=1 << 16)
    assert need(total_q=64, **many) > 0
    assert need(total_q=1 << 25, **many) == 0


def test_binding_refuses_host_tensors_and_bad_shapes():
    z = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    cfg = fq.make_cfg()
    with pytest.raises(ValueError, match="device tensors"):
        fq.KVCache(z(4, 2, 16, 32), z(4, 2, 16, 4), z(4, 2, 16, 32), z(4, 2, 16, 4), cfg)
    with pytest.raises(ValueError, match="k_scales"):
        fq.KVCache(z(4, 2, 16, 32), z(4, 2, 16, 2), z(4, 2, 16, 32), z(4, 2, 16, 4), cfg)
    with pytest.raises(ValueError, match="tensorwise"):
        fq.KVCache(z(4, 2, 16, 32), z(4, 2, 16, 4), z(4, 2, 16, 32), z(4, 2, 16, 4), cfg, k_outer=torch.ones(2),
                   v_outer=torch.ones(2))


def linear(cfg=None, x=FAKE, M=3, ld_x=128, codes=FAKE, scales=FAKE, outer=None, t=0, N=64, K=128, y=FAKE, ld_y=64, ws=None, wsb=0):
    cfg = cfg if cfg is not None else fq.make_cfg()
    return status(fq.lib().fp4_linear(ct.byref(cfg), x, M, ld_x, codes, scales, outer, t, N, K, y, ld_y, ws, wsb,
                                         None))


@no_gpu
def test_linear_rules():
    C = fq.make_cfg
    for kw in (dict(M=-1), dict(N=-1), dict(K=-32), dict(K=48), dict(ld_x=120), dict(ld_y=63)):
        assert linear(**kw) == fq.ERR_SHAPE, kw
    one_d, two_d = (C(two_level="outer_block", outer_block_size=n, outer_2d=b) for n, b in ((64, False), (64, True)))
    assert linear(cfg=one_d, K=96, ld_x=96, outer=FAKE) == fq.ERR_SHAPE
    assert linear(cfg=two_d, N=32, outer=FAKE) == fq.ERR_SHAPE
    assert linear(cfg=one_d) == fq.ERR_NULL and linear(cfg=two_d) == fq.ERR_NULL
    assert linear(cfg=C(two_level="tensorwise")) == fq.ERR_NULL
    for n, b in ((16, False), (32, False), (128, True)):
        assert linear(cfg=C(two_level="outer_block", outer_block_size=n, outer_2d=b), N=128, ld_y=128,
                      outer=FAKE) == fq.ERR_UNSUPPORTED
    assert linear(cfg=one_d, outer=FAKE, t=1) == fq.ERR_MODE and linear(t=2) == fq.ERR_MODE
    assert linear(cfg=C(input_dtype="fp32")) == fq.ERR_UNSUPPORTED
    assert linear(cfg=C(input_dtype="fp16")) == fq.ERR_DTYPE
    for kw in (dict(M=(1 << 20) + 1), dict(N=(1 << 24) + 1, ld_y=1 << 25), dict(K=(1 << 22) + 32, ld_x=1 << 23)):
        assert linear(**kw) == fq.ERR_UNSUPPORTED, kw
    for n in ("x", "codes", "scales", "y"):
        assert linear(**{n: None}) == fq.ERR_NULL
    for n in ("x", "codes"):
        assert linear(**{n: MIS}) == fq.ERR_ALIGN
    assert linear(y=FAKE + 1) == fq.ERR_ALIGN and linear(ld_x=132) == fq.ERR_ALIGN
    assert linear(cfg=C(two_level="tensorwise"), outer=FAKE + 2) == fq.ERR_ALIGN
    assert linear(scales=FAKE + 1) == fq.ERR_ALIGN
    assert linear(ld_x=(1 << 23) + 8) == fq.ERR_UNSUPPORTED
    big = dict(M=40, N=256, K=8192, ld_x=8192, ld_y=256)
    need = fq.fp4q_linear_workspace_bytes(40, 256, 8192)
    assert need > 0 and linear(**big) == fq.ERR_WORKSPACE and linear(ws=FAKE, wsb=need - 1, **big) == fq.ERR_WORKSPACE
    assert linear(ws=MIS, wsb=need, **big) == fq.ERR_ALIGN
    assert fq.fp4q_linear_workspace_bytes(-1, 256, 8192) == 0
    assert linear(M=0, x=None, y=None) == fq.OK and linear(N=0, codes=None, y=None) == fq.OK


def test_linear_binding_rules():
    u8 = torch.zeros(4, 16, dtype=torch.uint8)
    w = {"codes": u8, "scales": u8, "outer": None}
    with pytest.raises(fq.Fp4Error):
        fq.fp4_linear(torch.zeros(2, 32), w, fq.make_cfg())
    with pytest.raises(ValueError, match="disagree on K"):
        fq.fp4_linear(torch.zeros(2, 64, dtype=torch.bfloat16), w, fq.make_cfg())
    with pytest.raises(ValueError, match="device tensors"):
        fq.fp4_linear(torch.zeros(2, 32, dtype=torch.bfloat16), w, fq.make_cfg())
