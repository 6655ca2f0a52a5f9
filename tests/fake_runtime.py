"""The library over a CUDA runtime without a GPU (tests/host/fake_cuda.cpp): its own objects, linked with functions that
write launches to a log.  Pointers are numbers that nothing follows."""
import ctypes as C
import glob
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CUDA = os.environ.get("CUDA_HOME", "/usr/local/cuda")


def build(folder):
    import attention_frame_decode_b200 as vc
    objects = glob.glob(os.path.join(ROOT, "_build", "*.cu.o"))
    sources = glob.glob(os.path.join(ROOT, "attention_frame_decode_b200", "csrc", "*.cu"))
    if len(objects) < len(sources) or shutil.which("g++") is None or not os.path.isdir(CUDA):
        pytest.skip("needs the library's objects, g++ and the CUDA headers")
    so = os.path.join(str(folder), "libvc_fake.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-Wall", "-Wextra", "-Wl,-Bsymbolic", "-Wl,-z,defs",
                    "-I" + os.path.join(CUDA, "include"), "-o", so, os.path.join(HERE, "host", "fake_cuda.cpp")] +
                   [os.path.join(ROOT, "_build", os.path.basename(s) + ".o") for s in sources], check=True, timeout=300)
    lib, real = C.CDLL(so), vc.lib()
    for name in vc.EXPORTS:
        getattr(lib, name).argtypes, getattr(lib, name).restype = getattr(real, name).argtypes, getattr(real, name).restype
    lib.fake_log.restype = C.c_char_p
    lib.fake_fail.argtypes = [C.c_char_p, C.c_int, C.c_int]
    return lib


class Host:
    """a backbone whose calls end at the fake runtime"""

    def __init__(self, lib, cfg, max_batch=2, kv_capacity=64, n_slots=3, page=16, columns=8):
        import attention_frame_decode_b200 as vc
        import synth
        self.vc, self.lib, self.cfg, self.n_slots = vc, lib, cfg, n_slots
        self.at = 1 << 20
        layers = (vc.VcLayerWeights * cfg.n_layers)()
        for layer, kind in zip(layers, cfg.pattern):
            for f, t in vc.VcLayerWeights._fields_:
                if t is C.c_void_p:
                    setattr(layer, f, self.pointer())
        names = {synth.K_IN: "in_proj", synth.K_OUT: "out_proj", synth.K_QKV: "qkv", synth.K_O: "o", synth.K_UP: "up",
                 synth.K_DOWN: "down"}
        mat = lambda fmt, N, K: vc.VcQmat(self.pointer(), fmt, cfg.group_size, N, K)  # noqa: E731
        for l in range(cfg.n_layers):
            for kind, N, K in synth.linear_shapes(cfg, l):
                setattr(layers[l], names[kind], mat(cfg.wfmt, N, K))
        self.keep = layers
        self.w = vc.VcWeights(layers, self.pointer(), mat(cfg.head_fmt, cfg.vocab_text, cfg.d_model),
                              mat(cfg.head_fmt, cfg.vocab_func, cfg.d_model))
        self.c = vc.make_config(cfg, max_batch, kv_capacity, n_slots)
        self.h = C.c_void_p()
        lib.fake_reset()
        n = lib.vc_workspace_bytes(C.byref(self.c))
        assert lib.vc_backbone_create(C.byref(self.c), C.byref(self.w), self.pointer(), n, None, C.byref(self.h)) == vc.VC_OK
        self.state = vc.VcState(*[self.pointer() for _ in range(6)])
        kv = vc.VcPagedKv()
        for f in ("k", "v", "table", "len", "refs", "status", "workspace"):
            setattr(kv, f, self.pointer())
        kv.layers, kv.pages, kv.page_size = cfg.pattern.count("*"), 32, page
        kv.kv_heads, kv.head_dim, kv.q_heads = cfg.attn_kv_heads, cfg.attn_head_dim, cfg.attn_q_heads
        kv.seqs, kv.columns, kv.window, kv.sinks = n_slots, columns, 40, 2
        kv.workspace_bytes = lib.vc_paged_workspace_bytes(C.byref(kv))
        self.kv = kv
        self.x, self.tt, self.tf, self.slots = (self.pointer() for _ in range(4))
        lib.fake_reset()

    def pointer(self):
        self.at += 1 << 16
        return self.at

    def step(self, slots=False, B=2, emb=None):
        return self.lib.vc_step_paged(self.h, self.x, emb, B, self.slots if slots else None, C.byref(self.state),
                                      C.byref(self.kv), self.tt, self.tf, None)

    def prefill(self, T=20, slot=0):
        return self.lib.vc_prefill_paged(self.h, self.x, T, slot, C.byref(self.state), C.byref(self.kv), None)

    def option(self, option, value):
        assert self.lib.vc_set_option(self.h, option, value) == self.vc.VC_OK

    def fail(self, function, nth, error=2):
        self.lib.fake_fail(function.encode(), nth, error)

    def launches(self):
        """what has run since the last call of this"""
        out = self.lib.fake_log().decode().splitlines()
        self.lib.fake_reset()
        return out

    def close(self):
        self.lib.vc_destroy(self.h)
