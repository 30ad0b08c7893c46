"""Plans of the block's operators for a device that is not the current one
(CPU): block_plan_devices.cpp holds their plan layer against two devices that it
makes up."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "warp_specialized_pipelined_amd", "csrc")


def test_a_plan_prepares_its_own_device(tmp_path):
    exe = str(tmp_path / "block_plan_devices")
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    # (What a plan's creation does not call, launches above all, stays undefined.)
    subprocess.run(["g++", "-w", "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(rocm, "include"),
                    os.path.join(ROOT, "tests", "block_plan_devices.cpp"),
                    os.path.join(CSRC, "operators", "block_api.cpp"), "-o", exe,
                    "-Wl,--unresolved-symbols=ignore-all"], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout == "block_plan_devices: OK\n", (r.returncode, r.stdout, r.stderr)
