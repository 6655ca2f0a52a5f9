"""What the backbone's calls over a paged cache launch, and what they leave behind when the CUDA runtime fails, on a
runtime without a GPU."""
import pytest

import fake_runtime
import synth


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    return fake_runtime.build(tmp_path_factory.mktemp("fake"))


@pytest.fixture
def host(lib):
    h = fake_runtime.Host(lib, synth.tiny_config())
    yield h
    h.close()


def plain(x):
    return x.split("<")[0].split(" ")[0]


@pytest.mark.parametrize("slots", [False, True])
def test_a_step_asks_for_its_positions_first(host, slots):
    assert host.step(slots) == host.vc.VC_OK
    first = host.launches()
    names = [plain(x) for x in first]
    assert names[:3 + slots] == ["step_slots_kernel"] * slots + ["paged_resize_kernel", "paged_copy_kernel", "input_kernel"]
    assert names.count("paged_frame_kernel") == host.cfg.pattern.count("*")
    assert host.step(slots) == host.vc.VC_OK and host.launches() == first      # from the graph that is there
    host.option(host.vc.OPT_GRAPH, 0)
    assert host.step(slots) == host.vc.VC_OK and host.launches() == first      # directly


def test_any_tensor_of_slots_goes_with_one_graph(host):
    assert host.step(slots=True) == host.vc.VC_OK
    host.launches()
    host.slots = host.pointer()
    host.fail("cudaStreamBeginCapture", 1)
    assert host.step(slots=True) == host.vc.VC_OK and len(host.launches()) > 4


@pytest.mark.parametrize("function,nth", [("cudaStreamBeginCapture", 1), ("cudaLaunchKernel", 1), ("cudaLaunchKernel", 2),
                                          ("cudaLaunchKernelExC", 1), ("cudaLaunchKernelExC", 4),
                                          ("cudaLaunchKernelExC", 9), ("cudaFuncSetAttribute", 2), ("cudaStreamEndCapture", 1),
                                          ("cudaGraphInstantiate", 1), ("cudaGraphLaunch", 1)])
@pytest.mark.parametrize("slots", [False, True])
def test_a_step_that_fails_on_the_host_touches_no_session(host, function, nth, slots):
    """no length is one ahead of its session: the same call can be made again"""
    host.fail(function, nth)
    assert host.step(slots) == host.vc.VC_ERR_CUDA
    assert [x for x in host.launches() if x != "step_slots_kernel"] == []
    assert host.step(slots) == host.vc.VC_OK
    assert "paged_resize_kernel" in host.launches()


@pytest.mark.parametrize("shape", [dict(ssm_head_dim=12, ssm_heads=32), dict(ssm_state=20)], ids=str)
def test_a_prefill_of_shapes_that_it_does_not_cover_runs_nothing(lib, shape):
    h = fake_runtime.Host(lib, synth.tiny_config(**shape))
    assert h.prefill() == h.vc.VC_ERR_UNSUPPORTED and h.launches() == []
    assert h.lib.vc_prefill(h.h, h.x, 20, 0, h.state, None) == h.vc.VC_ERR_UNSUPPORTED and h.launches() == []
    h.close()


@pytest.mark.parametrize("nth", [6, 12, 20])
def test_a_prefill_that_fails_between_launches_has_taken_the_slots_frames(host, nth):
    """the slot's count is cleared before its pages change hands, and set by the last launch: no step takes it in between"""
    assert host.prefill() == host.vc.VC_OK
    names = [plain(x) for x in host.launches()]
    assert names.index("pf_paged_args_kernel") < names.index("paged_resize_kernel")
    assert names[-1] == "pf_paged_finish_kernel" and names.count("pf_paged_finish_kernel") == 1
    host.fail("cudaLaunchKernel", nth)
    assert host.prefill() == host.vc.VC_ERR_CUDA
    assert "pf_paged_finish_kernel" not in [plain(x) for x in host.launches()]


@pytest.mark.parametrize("graph", [0, 1])
def test_programmatic_launches_are_an_option(host, graph):
    """VC_OPT_PDL 0: no launch of a step or a prefill over a paged cache begins before the one before it ends"""
    host.option(host.vc.OPT_GRAPH, graph)
    for value in (0, 1):
        host.option(host.vc.OPT_PDL, value)
        for call in (host.step, host.prefill):
            assert call() == host.vc.VC_OK
            early = {plain(x) for x in host.launches() if x.endswith(" pdl")}
            assert bool(early) == bool(value)
            assert {"paged_copy_kernel"} <= early if value else not early


@pytest.mark.parametrize("cfg", [synth.nano_config(), synth.tiny_config(attn_q_heads=8, attn_head_dim=64, ssm_heads=4)],
                         ids=["nano", "projection wider than the Mamba-2 rows"])
def test_a_dense_prefills_scratch_has_no_room_for_pages(cfg):
    """bytes of workspace a frame of kv_capacity costs: the prefill's buffers and the split attention's records.  A paged
    prefill's queries, keys and values lie over the Mamba-2 layers' rows where these are as wide"""
    import ctypes
    import attention_frame_decode_b200 as vc
    size = lambda cap: vc.lib().vc_workspace_bytes(ctypes.byref(vc.make_config(cfg, 1, cap, 1)))  # noqa: E731
    up = lambda n: -(-n // 128) * 128  # noqa: E731
    E, Cx, H, d = cfg.d_inner, cfg.conv_dim, cfg.ssm_heads, cfg.d_model
    q, kv = cfg.attn_q_heads * cfg.attn_head_dim, cfg.attn_kv_heads * cfg.attn_head_dim
    zx, rows = E + Cx + H, q + 2 * kv
    big = up(max(E, cfg.mlp_hidden, q))
    a_frame = 4 * d + 4 + 2 * up(d) + 2 * big + 2 * zx + 2 * (q if rows <= zx else rows) + 4 * Cx + 8 * H + 4 * E + 2 * Cx
    a_chunk = 6 * H * cfg.ssm_head_dim * cfg.ssm_state                 # of 256 frames
    a_split = 4 * cfg.attn_q_heads * (cfg.attn_head_dim + 2)           # of 32 frames
    n = 4096
    assert size(2 * n) - size(n) == n * a_frame + n // 256 * a_chunk + n // 32 * a_split
