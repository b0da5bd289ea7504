"""Refusals of the window's operators at the ends of their arguments, on a machine without a GPU."""
import ctypes

import pytest

import verify_weight_streaming_b200 as mr

A = ctypes.c_void_p(256)


@pytest.mark.parametrize("inter,code", [
    (2 ** 30, mr.MR_ERR_UNSUPPORTED), (2 ** 31 - 64, mr.MR_ERR_UNSUPPORTED), (2 ** 30 - 64, mr.MR_ERR_UNSUPPORTED),
    (2 ** 20 + 64, mr.MR_ERR_UNSUPPORTED), (-64, mr.MR_ERR_INVALID_ARG), (-(2 ** 31), mr.MR_ERR_INVALID_ARG),
    (-(2 ** 30), mr.MR_ERR_INVALID_ARG),
])
def test_moe_window_w4_inter(inter, code):
    """2 * inter is formed only for sizes that hold it."""
    assert mr.lib.moe_window_w4(A, 128, A, A, 4, A, 1 << 62, A, 1 << 62, A, 128, 2, 4, 8, 128, inter, 0, 64, mr.MR_F32, 0,
                                A, 1 << 62, None) == code


def moe_args(torch, workspace):
    bf = torch.bfloat16
    return dict(X=torch.zeros(2, 128, dtype=bf), ids=torch.zeros(2, 4, dtype=torch.int32), weights=torch.zeros(2, 4),
                Wup=torch.zeros(8, 128, 128, dtype=bf), Wdown=torch.zeros(8, 128, 64, dtype=bf), Y=torch.zeros(2, 128),
                workspace=workspace)


def scattered(torch, size):
    """Workspaces that count more bytes than lie behind their address, or other ones."""
    return (torch.zeros(2 * size, dtype=torch.uint8)[::2], torch.zeros(1, dtype=torch.uint8).expand(size),
            torch.zeros((256, -(-size // 256)), dtype=torch.uint8).t())


def test_moe_window_refuses_a_scattered_workspace():
    torch = pytest.importorskip("torch")
    for ws in scattered(torch, mr.moe_window_workspace_bytes(2, 4, 128, 64)):
        args = moe_args(torch, ws)
        with pytest.raises(ValueError, match="workspace"):
            mr.moe_window_bf16(**args)
        del args["Wup"], args["Wdown"]
        packed = torch.zeros(8 * mr.w4_packed_bytes(128, 128, 64, True), dtype=torch.uint8)
        with pytest.raises(ValueError, match="workspace"):
            mr.moe_window_w4(up=packed, down=packed, experts=8, inter=64, fmt=64, **args)


def test_router_refuses_a_scattered_workspace():
    torch = pytest.importorskip("torch")
    bf = torch.bfloat16
    for ws in scattered(torch, mr.router_gemv_topk_workspace_bytes(2, 64, False)):
        with pytest.raises(ValueError, match="workspace"):
            mr.router_gemv_topk(torch.zeros(2, 128, dtype=bf), torch.zeros(64, 128, dtype=bf), 4,
                                torch.zeros(2, 4, dtype=torch.int32), workspace=ws, stream=0)


@pytest.mark.parametrize("group", [256, 288, 320, 384, 640, 896, 1024 + 128, 2 ** 16 + 64, -128, -1])
def test_group_sizes_that_no_format_word_holds(group):
    """Added to the flag bits they would be another format: 384 = 128 with zero points, 640 = 128 with f16 scales."""
    torch = pytest.importorskip("torch")
    for zeros in (False, True):
        for dtype in (torch.bfloat16, torch.float16):
            with pytest.raises(ValueError, match="group"):
                mr.w4_format(group, zeros, dtype)


def test_pack_refuses_one_group_a_row_that_is_too_long():
    """The scales of a 384-long group would be read as three groups' of 128, past their end."""
    torch = pytest.importorskip("torch")
    for k, dtype, zeros in ((384, torch.bfloat16, True), (640, torch.float16, False), (288, torch.bfloat16, True),
                            (896, torch.float16, True)):
        q, s = torch.zeros(16, k // 2, dtype=torch.uint8), torch.zeros(16, 1, dtype=dtype)
        z = torch.zeros(16, 1, dtype=torch.uint8) if zeros else None
        with pytest.raises(ValueError, match="group"):
            mr.w4_pack(q, s, z, torch.zeros(1 << 16, dtype=torch.uint8))


def test_sizes_beyond_32_bits_are_refused():
    """The C entry points take int32: a larger size must not be cut to its low bits."""
    torch = pytest.importorskip("torch")
    new = lambda *shape, dtype=torch.float32: torch.empty(shape, dtype=dtype, device="meta")  # noqa: E731
    wide, bf, i32, u8 = 2 ** 32 + 5, torch.bfloat16, torch.int32, torch.uint8
    with pytest.raises(ValueError, match="32 bits"):
        mr.token_logprobs(new(1, wide), lse=new(1))
    with pytest.raises(ValueError, match="32 bits"):
        mr.token_logprobs(new(wide, 4), lse=new(wide))
    with pytest.raises(ValueError, match="32 bits"):
        mr.token_logprobs(new(1, 8), new(1, wide, dtype=i32), new(1, wide))
    with pytest.raises(ValueError, match="32 bits"):
        mr.mrgemv_w4(new(2, 128, dtype=bf), new(1 << 20, dtype=u8), new(2, wide), 128)
    with pytest.raises(ValueError, match="32 bits"):
        mr.mrgemv_w4(new(2 ** 32 + 2, 128, dtype=bf), new(1 << 20, dtype=u8), new(2 ** 32 + 2, 16), 128)
    with pytest.raises(ValueError, match="32 bits"):
        mr.w4_pack(new(2 ** 32 + 16, 64, dtype=u8), new(2 ** 32 + 16, 1, dtype=bf), None, new(1 << 20, dtype=u8))
    with pytest.raises(ValueError, match="32 bits"):
        mr.w4_pack(new(2 ** 32 + 1, 16, 64, dtype=u8), new(2 ** 32 + 1, 16, 1, dtype=bf), None, new(1 << 20, dtype=u8))
    args = moe_args(torch, torch.zeros(1 << 16, dtype=u8))
    for size in (lambda: mr.w4_packed_bytes(2 ** 32 + 16, 128, 128), lambda: mr.moe_window_workspace_bytes(1, 1, 2 ** 32 + 8, 8)):
        with pytest.raises(ValueError, match="32 bits"):
            size()
    for base in (2 ** 32, 2 ** 31, -(2 ** 32)):
        with pytest.raises(ValueError, match="32 bits"):
            mr.moe_window_bf16(expert_base=base, **args)
    del args["Wup"], args["Wdown"]
    packed = torch.zeros(1 << 20, dtype=u8)
    for bad in (dict(experts=2 ** 32 + 8), dict(inter=2 ** 32 + 64), dict(expert_base=2 ** 32)):
        with pytest.raises(ValueError, match="32 bits"):
            mr.moe_window_w4(up=packed, down=packed, fmt=64, **dict(dict(experts=8, inter=64), **bad), **args)
