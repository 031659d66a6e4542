"""The build command's flags (no compiler is run)."""
from rank_latent_kv_mlra_b200 import build


def test_device_code_is_stored_as_it_is():
    """Packed device code is unpacked by a process's first handle, 12 of its 31 ms."""
    assert "--no-compress" in build.nvcc_command()
    assert "--no-compress" in build.nvcc_command(ptxas_verbose=True)


def test_the_target_is_sm_100a_alone():
    cmd = build.nvcc_command()
    assert [a for a in cmd if a.startswith("arch=")] == ["arch=compute_100a,code=sm_100a"]
